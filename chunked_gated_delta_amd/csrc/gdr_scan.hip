// The sequential part of the head-gated delta rule: the state from chunk to chunk, and the outputs.
//
// Value columns are independent, so a workgroup of 4 wavefronts owns one (sequence, value head) and 16
// of its columns and walks the chunks.  Inside a chunk wavefront i owns token rows 16i .. 16i + 15 and
// the state's rows dk/4 i .. dk/4 (i + 1) - 1, in registers (fp32 matrix-core results).  Every A operand
// (K, Q, K^T, T', P) is used by exactly one wavefront and is loaded straight into its registers;
// what wavefronts exchange (the state, E, U: 16 columns each) goes through LDS as ready B operands:
//   E = V - gam K S  |  U = beta T' E  |  O = scale gam Q S + P U,  S <- e^{G_last} S + K^T (eta U)
// with one barrier at each bar.  The state is an fp32 sum; as an operand it is hi + lo.
// The backward runs the same kernel without outputs: it leaves each chunk's entering state and F, which
// the gradient kernel reads (rounded to the inputs' type there: they enter gradients of that type).
#include "gdr_internal.h"

namespace kda {

namespace {

template <typename T, int DK, bool STATES>
__global__ __launch_bounds__(256) void gdr_scan_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  using Op = typename Frags<T>::Op;
  constexpr int KS = DK / 32;
  constexpr int RT = DK >= 64 ? DK / 64 : 1;      // state row tiles of a wavefront
  constexpr int kInFrag = Frags<T>::kInPlanes * kPlane, kOpFrag = 2 * kPlane;
  __shared__ __attribute__((aligned(16))) char sf[KS * kOpFrag];   // the state, as B operands
  __shared__ __attribute__((aligned(16))) char ef[2 * kOpFrag];    // E
  __shared__ __attribute__((aligned(16))) char uf[2 * kOpFrag];    // U
  __shared__ __attribute__((aligned(16))) char wf[2 * kOpFrag];    // eta U

  int64_t unit;
  int part;
  if (!gdr_block(blockIdx.x, p.n_seq * p.Hv, p.dv / 16, &unit, &part)) return;
  const int64_t s = unit / p.Hv;
  const int h = (int)(unit % p.Hv), kh = h / (p.Hv / p.Hk);
  const GdrSeq seq = gdr_seq(p, s);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  const int col = 16 * part + li;
  const bool owner = wave * RT < DK / 16;
  const int r0 = 16 * wave + 4 * g;               // first of this lane's 4 token rows in result tiles

  floatx4 S[RT];
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    S[m] = floatx4{};
    if (owner && p.S0) {
      const float* at = p.S0 + unit * p.dk * p.dv + (int64_t)(16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
      for (int r = 0; r < 4; ++r) S[m][r] = at[r * p.dv];
    }
  }
  auto put_state = [&]() {
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      const int t = wave * RT + m;
      if (owner) put_op(sf + (t >> 1) * kOpFrag, t & 1, li, g, S[m], T{});
    }
  };
  put_state();
  block_barrier();

  const T* kp = (const T*)p.k + seq.row * p.sk.b + kh * p.sk.h + (seq.t0 + 16 * wave + li) * p.sk.t + 8 * g;
  const T* qp = (const T*)p.q + seq.row * p.sq.b + kh * p.sq.h + (seq.t0 + 16 * wave + li) * p.sq.t + 8 * g;
  const T* vp = (const T*)p.v + seq.row * p.sv.b + h * p.sv.h + (seq.t0 + r0) * p.sv.t + col;
  T* op = STATES ? nullptr : (T*)p.o + seq.row * p.so.b + h * p.so.h + (seq.t0 + r0) * p.so.t + col;

  for (int64_t c = 0; c < seq.n_chunks; ++c) {
    const int64_t slot = seq.slot0 + c, blk = slot * p.Hv + h;
    const int64_t left = seq.len - c * kGdrChunk;
    const int n = left < kGdrChunk ? (int)left : kGdrChunk;
    const float* gate = (const float*)p.ws_gate + blk * kGateFloats;
    const floatx4 gam = ld4f(gate + kGateGam + r0), eta = ld4f(gate + kGateEta + r0), beta = ld4f(gate + kGateBeta + r0);
    const float last = gate[kGateLast];

    if constexpr (STATES) {   // the state entering the chunk
      if (owner) {
        T* at = (T*)p.ws_s + blk * p.dk * p.dv + (int64_t)(16 * wave * RT + 4 * g) * p.dv + col;
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) store_f32(at, (int64_t)(16 * m + r) * p.dv, S[m][r]);
      }
    }
    floatx4 E = {}, O = {};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      In kf, qf;
      zero_frag(kf);
      zero_frag(qf);
      if (16 * wave + li < n) {
        kf = load_row8(kp + c * kGdrChunk * p.sk.t + 32 * ks);
        if constexpr (!STATES) qf = load_row8(qp + c * kGdrChunk * p.sq.t + 32 * ks);
      }
      const Op b = load_frag<Op>(sf + ks * kOpFrag, lane);
      E = mma(kf, b, E);
      if constexpr (!STATES) O = mma(qf, b, O);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float v = r0 + r < n ? load_f32(vp, (c * kGdrChunk + r) * p.sv.t) : 0.f;
      E[r] = v - gam[r] * E[r];
    }
    put_op(ef + (wave >> 1) * kOpFrag, wave & 1, li, g, E, T{});
    block_barrier();

    floatx4 F = {};
    const char* ti = p.ws_ti + blk * kTriFrags * kOpFrag;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks <= wave / 2) F = mma(load_frag<Op>(ti + lower_frag(wave, ks) * kOpFrag, lane), load_frag<Op>(ef + ks * kOpFrag, lane), F);
    if constexpr (STATES) {
      T* at = (T*)p.ws_f + blk * kGdrChunk * p.dv + (int64_t)r0 * p.dv + col;
#pragma unroll
      for (int r = 0; r < 4; ++r) store_f32(at, (int64_t)r * p.dv, F[r]);
    }
    const floatx4 U = beta * F;
    if constexpr (!STATES) put_op(uf + (wave >> 1) * kOpFrag, wave & 1, li, g, U, T{});
    put_op(wf + (wave >> 1) * kOpFrag, wave & 1, li, g, eta * U, T{});
    block_barrier();

    if constexpr (!STATES) {
#pragma unroll
      for (int r = 0; r < 4; ++r) O[r] *= p.scale * gam[r];
      const char* pm = p.ws_p + blk * kTriFrags * kInFrag;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks <= wave / 2) O = mma(load_frag<In>(pm + lower_frag(wave, ks) * kInFrag, lane), load_frag<Op>(uf + ks * kOpFrag, lane), O);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < n) store_f32(op, (c * kGdrChunk + r) * p.so.t, O[r]);
    }
    if (owner) {
      const char* kt = p.ws_kt + (slot * p.Hk + kh) * (int64_t)(DK / 8) * kInFrag;
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        S[m] = S[m] * last;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          S[m] = mma(load_frag<In>(kt + (2 * (wave * RT + m) + ks) * kInFrag, lane), load_frag<Op>(wf + ks * kOpFrag, lane), S[m]);
      }
    }
    put_state();
    block_barrier();
  }

  if (p.S_final && owner) {
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      float* at = p.S_final + unit * p.dk * p.dv + (int64_t)(16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
      for (int r = 0; r < 4; ++r) at[r * p.dv] = S[m][r];
    }
  }
}

// The adjoint's sequential part, from the last chunk to the first, in the same division of work:
//   X = P^T dO + eta K dS  |  dU = T^T X, dE = beta dU (the gradient of v)
//   |  dS <- e^{G_last} dS + Q^T (scale gam dO) - K^T (gam dE)
// It leaves dS of each chunk's end for the gradient kernel and, per 16 columns, the sums of dU F that
// make beta's gradient.
template <typename T, int DK>
__global__ __launch_bounds__(256) void gdr_rscan_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  using Op = typename Frags<T>::Op;
  constexpr int KS = DK / 32;
  constexpr int RT = DK >= 64 ? DK / 64 : 1;
  constexpr int kInFrag = Frags<T>::kInPlanes * kPlane, kOpFrag = 2 * kPlane;
  __shared__ __attribute__((aligned(16))) char sf[KS * kOpFrag];   // dS
  __shared__ __attribute__((aligned(16))) char of[2 * kInFrag];    // dO
  __shared__ __attribute__((aligned(16))) char gf[2 * kOpFrag];    // scale gam dO
  __shared__ __attribute__((aligned(16))) char xf[2 * kOpFrag];    // X
  __shared__ __attribute__((aligned(16))) char ef[2 * kOpFrag];    // -gam dE

  int64_t unit;
  int part;
  if (!gdr_block(blockIdx.x, p.n_seq * p.Hv, p.dv / 16, &unit, &part)) return;
  const int64_t s = unit / p.Hv;
  const int h = (int)(unit % p.Hv), kh = h / (p.Hv / p.Hk);
  const GdrSeq seq = gdr_seq(p, s);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  const int col = 16 * part + li;
  const bool owner = wave * RT < DK / 16;
  const int r0 = 16 * wave + 4 * g;

  floatx4 S[RT];
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    S[m] = floatx4{};
    if (owner && p.dSf) {
      const float* at = p.dSf + unit * p.dk * p.dv + (int64_t)(16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
      for (int r = 0; r < 4; ++r) S[m][r] = at[r * p.dv];
    }
  }
  const T* kp = (const T*)p.k + seq.row * p.sk.b + kh * p.sk.h + (seq.t0 + 16 * wave + li) * p.sk.t + 8 * g;
  const T* dop = (const T*)p.dO + seq.row * p.sdo.b + h * p.sdo.h + (seq.t0 + r0) * p.sdo.t + col;
  T* dvp = (T*)p.dv_ + seq.row * p.sdv.b + h * p.sdv.h + (seq.t0 + r0) * p.sdv.t + col;

  for (int64_t c = seq.n_chunks - 1; c >= 0; --c) {
    const int64_t slot = seq.slot0 + c, blk = slot * p.Hv + h;
    const int64_t left = seq.len - c * kGdrChunk;
    const int n = left < kGdrChunk ? (int)left : kGdrChunk;
    const float* gate = (const float*)p.ws_gate + blk * kGateFloats;
    const floatx4 gam = ld4f(gate + kGateGam + r0), eta = ld4f(gate + kGateEta + r0), beta = ld4f(gate + kGateBeta + r0);
    const float last = gate[kGateLast];

    if (owner) {
      T* at = (T*)p.ws_ds + blk * p.dk * p.dv + (int64_t)(16 * wave * RT + 4 * g) * p.dv + col;
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const int t = wave * RT + m;
        put_op(sf + (t >> 1) * kOpFrag, t & 1, li, g, S[m], T{});
#pragma unroll
        for (int r = 0; r < 4; ++r) store_f32(at, (int64_t)(16 * m + r) * p.dv, S[m][r]);
      }
    }
    floatx4 dO;
#pragma unroll
    for (int r = 0; r < 4; ++r) dO[r] = r0 + r < n ? load_f32(dop, (c * kGdrChunk + r) * p.sdo.t) : 0.f;
    put_in(of + (wave >> 1) * kInFrag, wave & 1, li, g, dO, T{});
    put_op(gf + (wave >> 1) * kOpFrag, wave & 1, li, g, p.scale * (gam * dO), T{});
    block_barrier();

    floatx4 X = {};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      In kf;
      zero_frag(kf);
      if (16 * wave + li < n) kf = load_row8(kp + c * kGdrChunk * p.sk.t + 32 * ks);
      X = mma(kf, load_frag<Op>(sf + ks * kOpFrag, lane), X);
    }
    X = X * eta;
    const char* pm = p.ws_p + blk * kTriFrags * kOpFrag;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks >= wave / 2) X = mma(load_frag<Op>(pm + upper_frag(wave, ks) * kOpFrag, lane), load_frag<In>(of + ks * kInFrag, lane), X);
    put_op(xf + (wave >> 1) * kOpFrag, wave & 1, li, g, X, T{});
    block_barrier();

    floatx4 dU = {};
    const char* tt = p.ws_tt + blk * kTriFrags * kOpFrag;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks >= wave / 2) dU = mma(load_frag<Op>(tt + upper_frag(wave, ks) * kOpFrag, lane), load_frag<Op>(xf + ks * kOpFrag, lane), dU);
    const floatx4 dE = beta * dU;
    put_op(ef + (wave >> 1) * kOpFrag, wave & 1, li, g, -(gam * dE), T{});
    const T* fp = (const T*)p.ws_f + blk * kGdrChunk * p.dv + (int64_t)r0 * p.dv + col;
    float* db = (float*)p.ws_db + (blk * (p.dv / 16) + part) * kGdrChunk + r0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r0 + r < n) store_f32(dvp, (c * kGdrChunk + r) * p.sdv.t, dE[r]);
      float x = dU[r] * load_f32(fp, (int64_t)r * p.dv);
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) x += __shfl_xor(x, d);
      if (li == 0) db[r] = x;
    }
    block_barrier();

    if (owner) {
      const char* kt = p.ws_kt + (slot * p.Hk + kh) * (int64_t)(DK / 8) * kInFrag;
      const char* qt = p.ws_qt + (slot * p.Hk + kh) * (int64_t)(DK / 8) * kInFrag;
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        S[m] = S[m] * last;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const int f = (2 * (wave * RT + m) + ks) * kInFrag;
          S[m] = mma(load_frag<In>(qt + f, lane), load_frag<Op>(gf + ks * kOpFrag, lane), S[m]);
          S[m] = mma(load_frag<In>(kt + f, lane), load_frag<Op>(ef + ks * kOpFrag, lane), S[m]);
        }
      }
    }
    block_barrier();   // gf and ef are read before the next chunk's writes
  }

  if (p.dS0 && owner) {
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      float* at = p.dS0 + unit * p.dk * p.dv + (int64_t)(16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
      for (int r = 0; r < 4; ++r) at[r * p.dv] = S[m][r];
    }
  }
}

template <typename T, int DK>
hipError_t launch_scan(const GdrParams& p, hipStream_t s, int kind) {
  const dim3 grid((unsigned)gdr_blocks(p.n_seq * p.Hv, p.dv / 16));
  if (kind == 0) hipLaunchKernelGGL((gdr_scan_kernel<T, DK, false>), grid, dim3(256), 0, s, p);
  else if (kind == 1) hipLaunchKernelGGL((gdr_scan_kernel<T, DK, true>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((gdr_rscan_kernel<T, DK>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const GdrParams& p, hipStream_t s, int kind) {
  switch (p.dk) {
    case 32: return launch_scan<T, 32>(p, s, kind);
    case 64: return launch_scan<T, 64>(p, s, kind);
    default: return launch_scan<T, 128>(p, s, kind);
  }
}

hipError_t launch_kind(const GdrParams& p, hipStream_t s, int kind) {
  return p.dtype == KDA_DTYPE_BF16 ? launch_t<uint16_t>(p, s, kind) : launch_t<float>(p, s, kind);
}

}  // namespace

hipError_t launch_gdr_scan(const GdrParams& p, hipStream_t s, bool states) { return launch_kind(p, s, states ? 1 : 0); }
hipError_t launch_gdr_rscan(const GdrParams& p, hipStream_t s) { return launch_kind(p, s, 2); }

}  // namespace kda
