// The sequential part of the head-gated delta rule: the state from chunk to chunk, and the outputs.
//
// Value columns are independent, so a workgroup owns one (sequence, value head) and 16 of its columns and
// walks the chunks:
//   E = V - gam K S  |  U = beta T' E  |  S <- e^{G_last} S + K^T (eta U)         O = scale gam Q S + P U
// with a barrier at each bar.  What bounds it is that chain: three products of 16 columns, each waiting
// for the one before, so everything else is kept off it.
//  - Wavefronts 0-3 walk the chain.  Wavefront i owns token rows 16i .. 16i + 15 and a quarter of the
//    state's rows, in registers (fp32 matrix-core results).  Wavefronts 4-7, one more on each SIMD, form the
//    outputs (or, in the backward's run, write out the entering states and F) in the chain's shadow.
//  - Every A operand (K, Q, K^T, T', P) has exactly one reader in the workgroup and is loaded straight into its
//    registers, for the chunk after the next as soon as this chunk's is used: two register buffers, the
//    loop unrolled by two.  Loads past the last chunk are clamped to it.
//  - What the wavefronts exchange (the state, E, U: 16 columns each) goes through LDS as ready B operands.
// Rows behind the sequence's end read its last row; their E is set to zero, so nothing of them reaches
// the state, and their outputs are not written.
#include "gdr_internal.h"

namespace kda {

namespace {

__device__ __forceinline__ int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

// Writes `rows` contraction places x 16 columns of a B-operand array (first planes) to row-major memory:
// a lane takes 8 columns of one place.
template <typename T>
__device__ __forceinline__ void write_rows(const char* frags, int frag_bytes, int rows, T* out, int64_t ld, int tid) {
  for (int i = tid; i < rows * 2; i += 256) {
    const int r = i >> 1, c0 = (i & 1) * 8;
    const char* fr = frags + (r >> 5) * frag_bytes;
    T x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = frag_at<T>(fr, r & 31, c0 + e);
    typename Frags<T>::In v;
    __builtin_memcpy(&v, x, sizeof(v));
    *reinterpret_cast<typename Frags<T>::In*>(out + (int64_t)r * ld + c0) = v;
  }
}

template <typename T, int DK, bool STATES>
__global__ __launch_bounds__(512) void gdr_scan_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  using Op3 = typename Frags<T>::template Op<3>;
  using Op2 = typename Frags<T>::template Op<2>;
  using Op1 = typename Frags<T>::template Op<1>;
  constexpr int KS = DK / 32;
  constexpr int RT = DK >= 64 ? DK / 64 : 1;      // state row tiles of a wavefront
  constexpr int kIn = in_frag<T>(), kOp1 = op_frag<T, 1>(), kOp2 = op_frag<T, 2>(), kOp3 = op_frag<T, 3>();
  __shared__ __attribute__((aligned(16))) char sf[KS * kOp3];              // the state, as B operands
  __shared__ __attribute__((aligned(16))) char ef[2 * kOp3];               // E
  __shared__ __attribute__((aligned(16))) char wf[2 * kOp3];               // eta U
  __shared__ __attribute__((aligned(16))) char uf[2 * kOp2];               // U (F where states are written)

  int64_t unit;
  int part;
  if (!gdr_block(blockIdx.x, p.n_seq * p.Hv, p.dv / 16, &unit, &part)) return;
  const int64_t s = unit / p.Hv;
  const int h = (int)(unit % p.Hv), kh = h / (p.Hv / p.Hk);
  const GdrSeq seq = gdr_seq(p, s);
  const int64_t nc = seq.n_chunks;
  const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
  const bool chain = threadIdx.x < 256;
  const int wave = (threadIdx.x >> 6) & 3;
  const int col = 16 * part + li;
  const int r0 = 16 * wave + 4 * g;               // first of this lane's 4 token rows in result tiles
  const int64_t blk0 = seq.slot0 * p.Hv + h;      // workspace block of chunk 0; the next is Hv further
  const float* gates = (const float*)p.ws_gate + blk0 * kGateFloats;
  auto clamp_chunk = [&](int64_t c) { return min64(c, nc - 1); };
  auto row_of = [&](int64_t c) { return seq.t0 + min64(c * kGdrChunk + 16 * wave + li, seq.len - 1); };

  if (chain) {
    const bool owner = wave * RT < DK / 16;
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
        if (owner) put_op<3>(sf + (t >> 1) * kOp3, t & 1, li, g, S[m], T{});
      }
    };
    put_state();
    block_barrier();

    const T* kp = (const T*)p.k + seq.row * p.sk.b + kh * p.sk.h + 8 * g;
    const T* vp = (const T*)p.v + seq.row * p.sv.b + h * p.sv.h + col;
    struct Buf {
      In k[KS];
      Op3 ti[2];
      In kt[RT][2];
      float v[4];
      floatx4 gam, eta, beta;
      float last;
    };
    auto load_k = [&](Buf& b, int64_t c) {
      const T* at = kp + row_of(c) * p.sk.t;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) b.k[ks] = load_row8(at + 32 * ks);
    };
    auto load_v = [&](Buf& b, int64_t c) {
#pragma unroll
      for (int r = 0; r < 4; ++r) b.v[r] = load_f32(vp, (seq.t0 + min64(c * kGdrChunk + r0 + r, seq.len - 1)) * p.sv.t);
      b.gam = ld4f(gates + c * p.Hv * kGateFloats + kGateGam + r0);
    };
    auto load_ti = [&](Buf& b, int64_t c) {
      const char* at = p.ws_ti + (blk0 + c * p.Hv) * kTriFrags * kOp3;
      b.ti[0] = load_frag<Op3>(at + lower_frag(wave, 0) * kOp3, lane);
      if (wave >= 2) b.ti[1] = load_frag<Op3>(at + lower_frag(wave, 1) * kOp3, lane);
      const float* gt = gates + c * p.Hv * kGateFloats;
      b.eta = ld4f(gt + kGateEta + r0);
      b.beta = ld4f(gt + kGateBeta + r0);
      b.last = gt[kGateLast];
    };
    auto load_kt = [&](Buf& b, int64_t c) {
      if (!owner) return;
      const char* at = p.ws_kt + ((seq.slot0 + c) * p.Hk + kh) * (int64_t)(DK / 8) * kIn;
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) b.kt[m][ks] = load_frag<In>(at + (2 * (wave * RT + m) + ks) * kIn, lane);
    };
    auto step = [&](Buf& b, int64_t c) {
      const int64_t left = seq.len - c * kGdrChunk, ahead = clamp_chunk(c + 2);
      const int n = left < kGdrChunk ? (int)left : kGdrChunk;
      floatx4 E = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) E = mma(b.k[ks], load_frag<Op3>(sf + ks * kOp3, lane), E);
      load_k(b, ahead);
#pragma unroll
      for (int r = 0; r < 4; ++r) E[r] = r0 + r < n ? b.v[r] - b.gam[r] * E[r] : 0.f;
      load_v(b, ahead);
      put_op<3>(ef + (wave >> 1) * kOp3, wave & 1, li, g, E, T{});
      block_barrier();

      floatx4 F = mma(b.ti[0], load_frag<Op3>(ef, lane), floatx4{});
      if (wave >= 2) F = mma(b.ti[1], load_frag<Op3>(ef + kOp3, lane), F);
      const floatx4 U = b.beta * F, W = b.eta * U;
      const float last = b.last;
      load_ti(b, ahead);
      put_op<3>(wf + (wave >> 1) * kOp3, wave & 1, li, g, W, T{});
      block_barrier();

      put_op<2>(uf + (wave >> 1) * kOp2, wave & 1, li, g, STATES ? F : U, T{});
      if (owner) {
        const Op3 w0 = load_frag<Op3>(wf, lane), w1 = load_frag<Op3>(wf + kOp3, lane);
#pragma unroll
        for (int m = 0; m < RT; ++m) S[m] = mma(b.kt[m][1], w1, mma(b.kt[m][0], w0, S[m] * last));
      }
      load_kt(b, ahead);
      put_state();
      block_barrier();
    };
    if (nc > 0) {
      Buf b0, b1;
      const int64_t second = clamp_chunk(1);
      load_k(b0, 0);
      load_v(b0, 0);
      load_ti(b0, 0);
      load_kt(b0, 0);
      load_k(b1, second);
      load_v(b1, second);
      load_ti(b1, second);
      load_kt(b1, second);
      for (int64_t c = 0; c < nc; c += 2) {
        step(b0, c);
        if (c + 1 < nc) step(b1, c + 1);
      }
    }
    if (p.S_final && owner) {
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        float* at = p.S_final + unit * p.dk * p.dv + (int64_t)(16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
        for (int r = 0; r < 4; ++r) at[r * p.dv] = S[m][r];
      }
    }
    return;
  }

  block_barrier();   // the first state
  if constexpr (STATES) {
    const int tid = threadIdx.x & 255;
    T* sp = (T*)p.ws_s + blk0 * p.dk * p.dv + 16 * part;
    T* fp = (T*)p.ws_f + blk0 * kGdrChunk * p.dv + 16 * part;
    for (int64_t c = 0; c < nc; ++c) {
      // the state that enters this chunk, F of the one before
      write_rows<T>(sf, kOp3, DK, sp + c * p.Hv * p.dk * p.dv, p.dv, tid);
      if (c > 0) write_rows<T>(uf, kOp2, kGdrChunk, fp + (c - 1) * p.Hv * kGdrChunk * p.dv, p.dv, tid);
      block_barrier();
      block_barrier();
      block_barrier();
    }
    if (nc > 0) write_rows<T>(uf, kOp2, kGdrChunk, fp + (nc - 1) * p.Hv * kGdrChunk * p.dv, p.dv, tid);
  } else {
    const T* qp = (const T*)p.q + seq.row * p.sq.b + kh * p.sq.h + 8 * g;
    T* op = (T*)p.o + seq.row * p.so.b + h * p.so.h + (seq.t0 + r0) * p.so.t + col;
    struct Buf {
      In q[KS];
      Op1 pm[2];
      floatx4 gam;
    };
    auto load_q = [&](Buf& b, int64_t c) {
      const T* at = qp + row_of(c) * p.sq.t;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) b.q[ks] = load_row8(at + 32 * ks);
      b.gam = ld4f(gates + c * p.Hv * kGateFloats + kGateGam + r0);
    };
    auto load_p = [&](Buf& b, int64_t c) {
      const char* at = p.ws_p + (blk0 + c * p.Hv) * kTriFrags * kOp1;
      b.pm[0] = load_frag<Op1>(at + lower_frag(wave, 0) * kOp1, lane);
      if (wave >= 2) b.pm[1] = load_frag<Op1>(at + lower_frag(wave, 1) * kOp1, lane);
    };
    floatx4 O = {};
    // the outputs of chunk c, whose U the chain has left
    auto finish = [&](Buf& b, int64_t c) {
      const int64_t left = seq.len - c * kGdrChunk;
      const int n = left < kGdrChunk ? (int)left : kGdrChunk;
      const Op2 u0 = load_frag<Op2>(uf, lane);
      if constexpr (sizeof(T) == 2) {
        O = mma(b.pm[0].p[0], u0, O);
        if (wave >= 2) O = mma(b.pm[1].p[0], load_frag<Op2>(uf + kOp2, lane), O);
      } else {
        O = mma(b.pm[0], u0, O);
        if (wave >= 2) O = mma(b.pm[1], load_frag<Op2>(uf + kOp2, lane), O);
      }
      load_p(b, clamp_chunk(c + 2));
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < n) store_f32(op, (c * kGdrChunk + r) * p.so.t, O[r]);
    };
    auto step = [&](Buf& b, Buf& before, int64_t c) {
      if (c > 0) finish(before, c - 1);
      O = floatx4{};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        // two planes: o is rounded to the inputs' type
        O = mma(b.q[ks], load_frag<Op2>(sf + ks * kOp3, lane), O);
      }
      O *= p.scale * b.gam;
      load_q(b, clamp_chunk(c + 2));
      block_barrier();
      block_barrier();
      block_barrier();
    };
    if (nc > 0) {
      Buf b0, b1;
      load_q(b0, 0);
      load_p(b0, 0);
      load_q(b1, clamp_chunk(1));
      load_p(b1, clamp_chunk(1));
      for (int64_t c = 0; c < nc; c += 2) {
        step(b0, b1, c);
        if (c + 1 < nc) step(b1, b0, c + 1);
      }
      if (nc & 1) finish(b0, nc - 1);
      else finish(b1, nc - 1);
    }
  }
}

// The adjoint's sequential part, from the last chunk to the first, in the same division of work:
//   X = P^T dO + eta K dS  |  dU = T^T X, dE = beta dU (the gradient of v)
//   |  dS <- e^{G_last} dS + Q^T (scale gam dO) - K^T (gam dE)
// Wavefronts 0-3 walk the chain; wavefronts 4-7 form P^T dO and Q^T (scale gam dO) of the chunk that comes
// next, which do not depend on it, and write out dS of each chunk's end for the gradient kernel.  The
// chain leaves, per 16 columns, the sums of dU F that make beta's gradient.
template <typename T, int DK>
__global__ __launch_bounds__(512) void gdr_rscan_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  using Op3 = typename Frags<T>::template Op<3>;
  constexpr int KS = DK / 32;
  constexpr int RT = DK >= 64 ? DK / 64 : 1;
  constexpr int kIn = in_frag<T>(), kOp3 = op_frag<T, 3>();
  __shared__ __attribute__((aligned(16))) char sf[KS * kOp3];              // dS
  __shared__ __attribute__((aligned(16))) char xf[2 * kOp3];               // X
  __shared__ __attribute__((aligned(16))) char ef[2 * kOp3];               // -gam dE
  __shared__ __attribute__((aligned(16))) char of[2 * kIn];                // dO
  __shared__ __attribute__((aligned(16))) char gf[2 * kOp3];               // scale gam dO
  __shared__ __attribute__((aligned(16))) float x0[2][4 * 256];            // P^T dO, result tiles [wave][lane][4]
  __shared__ __attribute__((aligned(16))) float d0[2][DK / 16 * 256];      // Q^T (scale gam dO)

  int64_t unit;
  int part;
  if (!gdr_block(blockIdx.x, p.n_seq * p.Hv, p.dv / 16, &unit, &part)) return;
  const int64_t s = unit / p.Hv;
  const int h = (int)(unit % p.Hv), kh = h / (p.Hv / p.Hk);
  const GdrSeq seq = gdr_seq(p, s);
  const int64_t nc = seq.n_chunks;
  const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
  const bool chain = threadIdx.x < 256;
  const int wave = (threadIdx.x >> 6) & 3;
  const int col = 16 * part + li;
  const int r0 = 16 * wave + 4 * g;
  const bool owner = wave * RT < DK / 16;
  const int64_t blk0 = seq.slot0 * p.Hv + h;
  const float* gates = (const float*)p.ws_gate + blk0 * kGateFloats;
  auto clamp_chunk = [&](int64_t c) { return c < 0 ? 0 : c; };

  if (chain) {
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
    auto put_state = [&]() {
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const int t = wave * RT + m;
        if (owner) put_op<3>(sf + (t >> 1) * kOp3, t & 1, li, g, S[m], T{});
      }
    };
    put_state();
    const T* kp = (const T*)p.k + seq.row * p.sk.b + kh * p.sk.h + 8 * g;
    T* dvp = (T*)p.dv_ + seq.row * p.sdv.b + h * p.sdv.h + (seq.t0 + r0) * p.sdv.t + col;
    struct Buf {
      In k[KS];
      Op3 tt[2];
      In kt[RT][2];
      float f[4];
      floatx4 gam, eta, beta;
      float last;
    };
    auto load_k = [&](Buf& b, int64_t c) {
      const T* at = kp + (seq.t0 + min64(c * kGdrChunk + 16 * wave + li, seq.len - 1)) * p.sk.t;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) b.k[ks] = load_row8(at + 32 * ks);
      b.eta = ld4f(gates + c * p.Hv * kGateFloats + kGateEta + r0);
    };
    auto load_tt = [&](Buf& b, int64_t c) {
      const char* at = p.ws_tt + (blk0 + c * p.Hv) * kTriFrags * kOp3;
      if (wave < 2) b.tt[0] = load_frag<Op3>(at + upper_frag(wave, 0) * kOp3, lane);
      b.tt[1] = load_frag<Op3>(at + upper_frag(wave, 1) * kOp3, lane);
      const float* gt = gates + c * p.Hv * kGateFloats;
      b.gam = ld4f(gt + kGateGam + r0);
      b.beta = ld4f(gt + kGateBeta + r0);
      b.last = gt[kGateLast];
    };
    auto load_kt = [&](Buf& b, int64_t c) {
      const T* fp = (const T*)p.ws_f + (blk0 + c * p.Hv) * kGdrChunk * p.dv + (int64_t)r0 * p.dv + col;
#pragma unroll
      for (int r = 0; r < 4; ++r) b.f[r] = load_f32(fp, (int64_t)r * p.dv);
      if (!owner) return;
      const char* at = p.ws_kt + ((seq.slot0 + c) * p.Hk + kh) * (int64_t)(DK / 8) * kIn;
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) b.kt[m][ks] = load_frag<In>(at + (2 * (wave * RT + m) + ks) * kIn, lane);
    };
    auto step = [&](Buf& b, int64_t c) {
      const int64_t left = seq.len - c * kGdrChunk, ahead = clamp_chunk(c - 2);
      const int n = left < kGdrChunk ? (int)left : kGdrChunk;
      floatx4 X = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) X = mma(b.k[ks], load_frag<Op3>(sf + ks * kOp3, lane), X);
      const floatx4 first = ld4f(&x0[c & 1][(wave * 64 + lane) * 4]);
#pragma unroll
      for (int r = 0; r < 4; ++r) X[r] = r0 + r < n ? b.eta[r] * X[r] + first[r] : 0.f;
      load_k(b, ahead);
      put_op<3>(xf + (wave >> 1) * kOp3, wave & 1, li, g, X, T{});
      block_barrier();

      floatx4 dU = mma(b.tt[1], load_frag<Op3>(xf + kOp3, lane), floatx4{});
      if (wave < 2) dU = mma(b.tt[0], load_frag<Op3>(xf, lane), dU);
      const floatx4 dE = b.beta * dU, G = -(b.gam * dE);
      const float last = b.last;
      load_tt(b, ahead);
      put_op<3>(ef + (wave >> 1) * kOp3, wave & 1, li, g, G, T{});
      block_barrier();

      if (owner) {
        const Op3 e0 = load_frag<Op3>(ef, lane), e1 = load_frag<Op3>(ef + kOp3, lane);
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          const floatx4 add = ld4f(&d0[c & 1][((wave * RT + m) * 64 + lane) * 4]);
          S[m] = mma(b.kt[m][1], e1, mma(b.kt[m][0], e0, S[m] * last + add));
        }
      }
      float* db = (float*)p.ws_db + ((blk0 + c * p.Hv) * (p.dv / 16) + part) * kGdrChunk + r0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r0 + r < n) store_f32(dvp, (c * kGdrChunk + r) * p.sdv.t, dE[r]);
        float x = dU[r] * b.f[r];
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) x += __shfl_xor(x, d);
        if (li == 0) db[r] = x;
      }
      load_kt(b, ahead);
      put_state();
      block_barrier();
    };
    block_barrier();
    block_barrier();
    if (nc > 0) {
      Buf b0, b1;
      const int64_t second = clamp_chunk(nc - 2);
      load_k(b0, nc - 1);
      load_tt(b0, nc - 1);
      load_kt(b0, nc - 1);
      load_k(b1, second);
      load_tt(b1, second);
      load_kt(b1, second);
      for (int64_t c = nc - 1; c >= 0; c -= 2) {
        step(b0, c);
        if (c > 0) step(b1, c - 1);
      }
    }
    if (p.dS0 && owner) {
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        float* at = p.dS0 + unit * p.dk * p.dv + (int64_t)(16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
        for (int r = 0; r < 4; ++r) at[r * p.dv] = S[m][r];
      }
    }
    return;
  }

  const int tid = threadIdx.x & 255;
  const T* dop = (const T*)p.dO + seq.row * p.sdo.b + h * p.sdo.h + col;
  T* sp = (T*)p.ws_ds + blk0 * p.dk * p.dv + 16 * part;
  struct Buf {
    float o[4];
    floatx4 gam;
    Op3 pm[2];
    In qt[RT][2];
  };
  auto load_o = [&](Buf& b, int64_t c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) b.o[r] = load_f32(dop, (seq.t0 + min64(c * kGdrChunk + r0 + r, seq.len - 1)) * p.sdo.t);
    b.gam = ld4f(gates + c * p.Hv * kGateFloats + kGateGam + r0);
  };
  auto load_pq = [&](Buf& b, int64_t c) {
    const char* at = p.ws_p + (blk0 + c * p.Hv) * kTriFrags * kOp3;
    if (wave < 2) b.pm[0] = load_frag<Op3>(at + upper_frag(wave, 0) * kOp3, lane);
    b.pm[1] = load_frag<Op3>(at + upper_frag(wave, 1) * kOp3, lane);
    if (!owner) return;
    const char* qt = p.ws_qt + ((seq.slot0 + c) * p.Hk + kh) * (int64_t)(DK / 8) * kIn;
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) b.qt[m][ks] = load_frag<In>(qt + (2 * (wave * RT + m) + ks) * kIn, lane);
  };
  auto spread = [&](Buf& b, int64_t c) {       // dO of chunk c as operands
    const int64_t left = seq.len - c * kGdrChunk;
    floatx4 o;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = r0 + r < left ? b.o[r] : 0.f;
    put_op<1>(of + (wave >> 1) * kIn, wave & 1, li, g, o, T{});
    put_op<3>(gf + (wave >> 1) * kOp3, wave & 1, li, g, p.scale * (b.gam * o), T{});
    load_o(b, clamp_chunk(c - 1));
  };
  auto products = [&](Buf& b, int64_t c) {
    floatx4 X = mma(b.pm[1], load_frag<In>(of + kIn, lane), floatx4{});
    if (wave < 2) X = mma(b.pm[0], load_frag<In>(of, lane), X);
    *reinterpret_cast<floatx4*>(&x0[c & 1][(wave * 64 + lane) * 4]) = X;
    if (owner) {
      const Op3 g0 = load_frag<Op3>(gf, lane), g1 = load_frag<Op3>(gf + kOp3, lane);
#pragma unroll
      for (int m = 0; m < RT; ++m)
        *reinterpret_cast<floatx4*>(&d0[c & 1][((wave * RT + m) * 64 + lane) * 4]) = mma(b.qt[m][1], g1, mma(b.qt[m][0], g0, floatx4{}));
    }
    load_pq(b, clamp_chunk(c - 1));
  };
  Buf b;
  if (nc > 0) {
    load_o(b, nc - 1);
    load_pq(b, nc - 1);
    spread(b, nc - 1);
  }
  block_barrier();
  if (nc > 0) products(b, nc - 1);
  block_barrier();
  for (int64_t c = nc - 1; c >= 0; --c) {
    // dS at this chunk's end; what the next one needs
    write_rows<T>(sf, kOp3, DK, sp + c * p.Hv * p.dk * p.dv, p.dv, tid);
    if (c > 0) spread(b, c - 1);
    block_barrier();
    if (c > 0) products(b, c - 1);
    block_barrier();
    block_barrier();
  }
}

template <typename T, int DK>
hipError_t launch_scan(const GdrParams& p, hipStream_t s, int kind) {
  const dim3 grid((unsigned)gdr_blocks(p.n_seq * p.Hv, p.dv / 16));
  if (kind == 0) hipLaunchKernelGGL((gdr_scan_kernel<T, DK, false>), grid, dim3(512), 0, s, p);
  else if (kind == 1) hipLaunchKernelGGL((gdr_scan_kernel<T, DK, true>), grid, dim3(512), 0, s, p);
  else hipLaunchKernelGGL((gdr_rscan_kernel<T, DK>), grid, dim3(512), 0, s, p);
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
