// Gradients of the head-gated delta rule from each chunk's entering state S, F = U / beta, the state's
// adjoint dS at the chunk's end and dE (the gradient of v): one workgroup per (chunk, key head), the
// value heads that share the key head one after another.
//
// Wavefront i owns the 16 tokens of tile i and forms the transposed gradients (channels x tokens), so a
// lane holds one token and 4 consecutive channels.  With dO' = scale dO and D_rj = e^{G_r - G_j}:
//   dP = lower(dO' U^T . D)   dA = -strict_lower(dE U^T . D)
//   dq_r  =  gam_r S dO'_r + sum_j dP_rj k_j
//   dk_r  = -gam_r S dE_r  + sum_j dA_rj k_j                                    (as a row: reads)
//         +  eta_r dS U_r  + sum_r' dA_r'r k_r' + sum_r' dP_r'r q_r'            (as a column: writes)
//   dG_r  = q_r . dq_r + k_r . dk_r(row) - k_r . dk_r(column),   dG_last += sum_r k_r . eta_r dS U_r + e^{G_last} <S, dS>
//   dg_t  = sum_{r >= t} dG_r
// The second identity gives the log-decay's gradient from the accumulators that are there anyway.  S,
// dS, F and dE are held in the inputs' type here (their rounding is one of the gradients' own size, half a
// step of that type); dP and dA take two planes, which keeps the error below 1.5 times the final rounding's.
#include "gdr_internal.h"

namespace kda {

namespace {

template <typename T, int DK, int DV>
__global__ __launch_bounds__(256) void gdr_grad_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  using Op = typename Frags<T>::template Op<2>;
  constexpr int KV = DV / 32, MT = DK / 16;
  constexpr int kInFrag = in_frag<T>(), kOpFrag = op_frag<T, 2>();
  __shared__ __attribute__((aligned(16))) char tri[4][4 * kOpFrag];   // a wavefront's dP and dA, two steps each
  __shared__ float ghi[64], glo[64], bet[64];
  __shared__ double dG[64];
  __shared__ double extra[4];

  GdrSeq seq;
  int64_t chunk;
  const int64_t slot = blockIdx.x;
  if (!gdr_find(p, slot, &seq, &chunk)) return;
  const int kh = blockIdx.y, grp = p.Hv / p.Hk;
  const int lane = threadIdx.x & 63, wave = wave_id(), li = lane & 15, g = lane >> 4;
  const int64_t t0 = seq.t0 + chunk * kGdrChunk, left = seq.len - chunk * kGdrChunk;
  const int n = left < kGdrChunk ? (int)left : kGdrChunk;
  const int tok = 16 * wave + li;                 // this lane's token
  const bool live = tok < n;
  char* dp_f = tri[wave];                         // dP (transposed, then as it is)
  char* da_f = tri[wave] + 2 * kOpFrag;

  const auto qrow = global_in<T>(p.q) + seq.row * p.sq.b + kh * p.sq.h + (t0 + tok) * p.sq.t + 4 * g;
  const auto krow = global_in<T>(p.k) + seq.row * p.sk.b + kh * p.sk.h + (t0 + tok) * p.sk.t + 4 * g;
  const auto kt = as_global((const char*)p.ws_kt) + (slot * p.Hk + kh) * (int64_t)(DK / 8) * kInFrag;
  const auto qt = as_global((const char*)p.ws_qt) + (slot * p.Hk + kh) * (int64_t)(DK / 8) * kInFrag;

  floatx4 dq[MT], dk[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) dq[m] = dk[m] = floatx4{};

  for (int hg = 0; hg < grp; ++hg) {
    const int h = kh * grp + hg;
    const int64_t blk = slot * p.Hv + h;
    const auto gate = global_in<float>(p.ws_gate) + blk * kGateFloats;
    if (wave == 0) {
      ghi[lane] = gate[kGateHi + lane];
      glo[lane] = gate[kGateLo + lane];
      bet[lane] = gate[kGateBeta + lane];
    }
    const float gam = gate[kGateGam + tok], eta = gate[kGateEta + tok], last = gate[kGateLast];
    const auto F = global_in<T>(p.ws_f) + blk * kGdrChunk * DV + 8 * g;
    const auto St = global_in<T>(p.ws_s) + blk * DK * DV + 8 * g;
    const auto dSt = global_in<T>(p.ws_ds) + blk * DK * DV + 8 * g;
    const auto dO = global_in<T>(p.dO) + seq.row * p.sdo.b + h * p.sdo.h + t0 * p.sdo.t + 8 * g;
    const auto dE = global_in<T>(p.dv_) + seq.row * p.sdv.b + h * p.sdv.h + t0 * p.sdv.t + 8 * g;
    auto f_frag = [&](int tile, int kv) { return load_row8(F + (int64_t)(16 * tile + li) * DV + 32 * kv); };
    auto rows_of = [&](GlobalPtr<const T> base, int64_t st, int tile, int kv) {
      In x;
      zero_frag(x);
      if (16 * tile + li < n) x = load_row8(base + (int64_t)(16 * tile + li) * st + 32 * kv);
      return x;
    };
    In fo[KV], oo[KV], eo[KV];   // this wavefront's own tokens
#pragma unroll
    for (int kv = 0; kv < KV; ++kv) {
      fo[kv] = f_frag(wave, kv);
      oo[kv] = rows_of(dO, p.sdo.t, wave, kv);
      eo[kv] = rows_of(dE, p.sdv.t, wave, kv);
    }
    __syncthreads();
    const float ghr = ghi[tok], glr = glo[tok], br = bet[tok];

    // rows: dP_rj and dA_rj of this wavefront's r over all j <= r, as B operands over j
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (m > (wave | 1)) continue;
      floatx4 a = {}, b = {};
      if (m <= wave) {
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) {
          const In f = f_frag(m, kv);
          a = mma(f, oo[kv], a);
          b = mma(f, eo[kv], b);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * m + 4 * g + r;
          const float d = tok >= j ? bet[j] * expf((ghr - ghi[j]) + (glr - glo[j])) : 0.f;
          a[r] = tok >= j ? p.scale * d * a[r] : 0.f;
          b[r] = tok > j ? -d * b[r] : 0.f;
        }
      }
      put_op<2>(dp_f + (m >> 1) * kOpFrag, m & 1, li, g, a, T{});
      put_op<2>(da_f + (m >> 1) * kOpFrag, m & 1, li, g, b, T{});
    }
    compiler_fence();
    double dg = 0.0, write = 0.0, hold = 0.0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      floatx4 a = {}, b = {};
      float ss = 0.f;
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
        const In st = load_row8(St + (int64_t)(16 * m + li) * DV + 32 * kv);
        a = mma(st, oo[kv], a);
        b = mma(st, eo[kv], b);
        if ((m & 3) == wave) {   // <S, dS>: every row tile once
          const In dst = load_row8(dSt + (int64_t)(16 * m + li) * DV + 32 * kv);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += (float)st[e] * (float)dst[e];
        }
      }
      hold += ss;
      a *= gam * p.scale;
      b *= -gam;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks > wave / 2) continue;
        const In x = load_frag<In>(kt + (2 * m + ks) * kInFrag, lane);
        a = mma(x, load_frag<Op>(dp_f + ks * kOpFrag, lane), a);
        b = mma(x, load_frag<Op>(da_f + ks * kOpFrag, lane), b);
      }
      dq[m] += a;
      dk[m] += b;
      if (live) {
        const floatx4 q4 = load_row4(qrow + 16 * m), k4 = load_row4(krow + 16 * m);
#pragma unroll
        for (int r = 0; r < 4; ++r) dg += (double)q4[r] * (double)a[r] + (double)k4[r] * (double)b[r];
      }
    }
    compiler_fence();

    // columns: dP_rj and dA_rj of this wavefront's j over all r >= j, as B operands over r
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (m < (wave & 2)) continue;
      floatx4 a = {}, b = {};
      if (m >= wave) {
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) {
          a = mma(rows_of(dO, p.sdo.t, m, kv), fo[kv], a);
          b = mma(rows_of(dE, p.sdv.t, m, kv), fo[kv], b);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * m + 4 * g + r;
          const float d = i >= tok ? br * expf((ghi[i] - ghr) + (glo[i] - glr)) : 0.f;
          a[r] = i >= tok ? p.scale * d * a[r] : 0.f;
          b[r] = i > tok ? -d * b[r] : 0.f;
        }
      }
      put_op<2>(dp_f + (m >> 1) * kOpFrag, m & 1, li, g, a, T{});
      put_op<2>(da_f + (m >> 1) * kOpFrag, m & 1, li, g, b, T{});
    }
    compiler_fence();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      floatx4 a = {};
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) a = mma(load_row8(dSt + (int64_t)(16 * m + li) * DV + 32 * kv), fo[kv], a);
      a *= eta * br;
      floatx4 k4 = {};
      if (live) k4 = load_row4(krow + 16 * m);
#pragma unroll
      for (int r = 0; r < 4; ++r) write += (double)k4[r] * (double)a[r];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks < wave / 2) continue;
        a = mma(load_frag<In>(kt + (2 * m + ks) * kInFrag, lane), load_frag<Op>(da_f + ks * kOpFrag, lane), a);
        a = mma(load_frag<In>(qt + (2 * m + ks) * kInFrag, lane), load_frag<Op>(dp_f + ks * kOpFrag, lane), a);
      }
      dk[m] += a;
#pragma unroll
      for (int r = 0; r < 4; ++r) dg -= (double)k4[r] * (double)a[r];
    }
    // the log-decay's gradient
    dg += __shfl_xor(dg, 16);
    dg += __shfl_xor(dg, 32);
    double ex = write + (double)last * hold;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) ex += __shfl_xor(ex, d);
    if (g == 0) dG[tok] = dg;
    if (lane == 0) extra[wave] = ex;
    __syncthreads();
    if (wave == 0) {
      double x = dG[lane];
      if (lane == 63) x += extra[0] + extra[1] + extra[2] + extra[3];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double dn = __shfl_down(x, d);
        if (lane + d < 64) x += dn;
      }
      if (lane < n) {
        const float w = get(global_in<T>(p.w) + seq.row * p.sw.b + h * p.sw.h + (t0 + lane) * p.sw.t);
        put(global_out<T>(p.dw) + seq.row * p.sdw.b + h * p.sdw.h + (t0 + lane) * p.sdw.t,
            (float)(x * (double)gdr_gate_grad(w, p.gate, p.g_min)));
        const auto db = global_in<float>(p.ws_db) + blk * (DV / 16) * kGdrChunk + lane;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) sum += db[c * kGdrChunk];
        put(global_out<T>(p.dbeta) + seq.row * p.sdb.b + h * p.sdb.h + (t0 + lane) * p.sdb.t, sum);
      }
    }
    __syncthreads();
  }

  if (live) {
    const auto dqp = global_out<T>(p.dq) + seq.row * p.sdq.b + kh * p.sdq.h + (t0 + tok) * p.sdq.t + 4 * g;
    const auto dkp = global_out<T>(p.dk_) + seq.row * p.sdk.b + kh * p.sdk.h + (t0 + tok) * p.sdk.t + 4 * g;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      store_row4(dqp + 16 * m, dq[m]);
      store_row4(dkp + 16 * m, dk[m]);
    }
  }
}

template <typename T, int DK>
hipError_t launch_dk(const GdrParams& p, hipStream_t s) {
  const dim3 grid((unsigned)gdr_slots(p.B, p.T, p.n_seq, p.seq_start != nullptr), (unsigned)p.Hk);
  if (grid.x == 0) return hipSuccess;
  switch (p.dv) {
    case 32: hipLaunchKernelGGL((gdr_grad_kernel<T, DK, 32>), grid, dim3(256), 0, s, p); break;
    case 64: hipLaunchKernelGGL((gdr_grad_kernel<T, DK, 64>), grid, dim3(256), 0, s, p); break;
    default: hipLaunchKernelGGL((gdr_grad_kernel<T, DK, 128>), grid, dim3(256), 0, s, p); break;
  }
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const GdrParams& p, hipStream_t s) {
  switch (p.dk) {
    case 32: return launch_dk<T, 32>(p, s);
    case 64: return launch_dk<T, 64>(p, s);
    default: return launch_dk<T, 128>(p, s);
  }
}

}  // namespace

hipError_t launch_gdr_grad(const GdrParams& p, hipStream_t s) {
  return p.dtype == KDA_DTYPE_BF16 ? launch_t<uint16_t>(p, s) : launch_t<float>(p, s);
}

}  // namespace kda
