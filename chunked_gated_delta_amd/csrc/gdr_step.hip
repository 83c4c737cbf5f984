// Recurrent step of the head-gated delta rule on a pool of resident states, a few tokens per row.
//
// Bound by the state's two trips through HBM.  A workgroup owns one (row, value head) and CB value
// columns; a thread holds 4 columns (one 16-byte access) of DK / RG consecutive state rows for all the
// call's tokens.  One decay per head lets both reductions run on the state as it was loaded:
//   a = S^T k,  b = S^T q,  d = k . q:   f = v - e^g a,  S <- e^g S + k (beta f)^T,  o = scale (e^g b + d beta f)
// so a token costs one exchange between the row groups (lanes by shuffles, wavefronts through LDS).
//
// 512 rows of 16 heads of 128 x 128: 1.07 GB in 221 us, 4.8 TB/s, a large copy's rate; one row of 8 heads: 5 us.
//
// Rows that name the same slot are successive tokens of that state: the first such row's workgroup
// takes them all in order and the others return, so no two workgroups touch one state.  Every workgroup reads
// all the slots for that, 4 bytes a row of the call beside the 32 KiB of its state's two trips.
#include "gdr_internal.h"

namespace kda {

namespace {

template <typename T, int DK, int CB>
__global__ __launch_bounds__(256) void gdr_step_kernel(GdrStepParams p) {
  constexpr int CT = CB / 4;             // threads along the columns
  constexpr int RG = 256 / CT;           // row groups
  constexpr int RPT = DK / RG;           // state rows of a thread
  constexpr int RW = 64 / CT;            // row groups of a wavefront
  static_assert(RPT >= 1 && RW >= 1, "tile");
  __shared__ __attribute__((aligned(16))) float part[2][4][2 * CB + 4];
  __shared__ int same[2];
  const int tid = threadIdx.x, ct = tid % CT, rg = tid / CT, wave = wave_id(), lane = tid & 63;
  const int nblk = p.dv / CB;
  const int64_t unit = blockIdx.x / nblk;
  const int64_t b0 = unit / p.Hv;
  const int h = (int)(unit % p.Hv), kh = h / (p.Hv / p.Hk);
  const int col = (int)(blockIdx.x % nblk) * CB + 4 * ct;

  const int64_t slot = p.slots ? p.slots[b0] : b0;
  if (slot < 0 || slot >= p.n_slots) {   // a padding row: zeros
    for (int64_t t = 0; t < p.T; ++t)
      if (rg == 0) store_row4(global_out<T>(p.o) + b0 * p.so.b + h * p.so.h + t * p.so.t + col, floatx4{});
    return;
  }
  const auto Sp = as_global(p.S) + (slot * p.Hv + h) * DK * (int64_t)p.dv + (int64_t)rg * RPT * p.dv + col;
  floatx4 S[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) S[i] = ld4f(Sp + (int64_t)i * p.dv);

  bool later = false;
  if (p.slots) {
    if (tid < 2) same[tid] = 0;
    __syncthreads();
    for (int64_t i = tid; i < p.B; i += 256)
      if (p.slots[i] == (int32_t)slot && i != b0) same[i > b0] = 1;
    __syncthreads();
    if (same[0]) return;
    later = same[1] != 0;
  }

  int phase = 0;
  for (int64_t b = b0; b < p.B; ++b) {
    if (b != b0 && p.slots[b] != (int32_t)slot) continue;
    for (int64_t t = 0; t < p.T; ++t) {
      const auto kp = global_in<T>(p.k) + b * p.sk.b + kh * p.sk.h + t * p.sk.t + rg * RPT;
      const auto qp = global_in<T>(p.q) + b * p.sq.b + kh * p.sq.h + t * p.sq.t + rg * RPT;
      const floatx4 v = load_row4(global_in<T>(p.v) + b * p.sv.b + h * p.sv.h + t * p.sv.t + col);
      const float decay = expf(gdr_gate(get(global_in<T>(p.w) + b * p.sw.b + h * p.sw.h + t * p.sw.t), p.gate, p.g_min));
      const float beta = get(global_in<T>(p.beta) + b * p.sb.b + h * p.sb.h + t * p.sb.t);
      float kk[RPT], qq[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        kk[i] = get(kp + i);
        qq[i] = get(qp + i);
      }
      floatx4 a = {}, o = {};
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        a += S[i] * kk[i];
        o += S[i] * qq[i];
        d += kk[i] * qq[i];
      }
#pragma unroll
      for (int m = CT; m < 64; m <<= 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          a[r] += __shfl_xor(a[r], m);
          o[r] += __shfl_xor(o[r], m);
        }
        d += __shfl_xor(d, m);
      }
      float* mine = part[phase][wave];
      if (lane < CT) {
        *reinterpret_cast<floatx4*>(mine + 4 * ct) = a;
        *reinterpret_cast<floatx4*>(mine + CB + 4 * ct) = o;
        if (lane == 0) mine[2 * CB] = d;
      }
      block_barrier();
      floatx4 sa = {}, so = {};
      float sd = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        sa += ld4f(part[phase][w] + 4 * ct);
        so += ld4f(part[phase][w] + CB + 4 * ct);
        sd += part[phase][w][2 * CB];
      }
      const floatx4 u = beta * (v - decay * sa);
      if (rg == 0) store_row4(global_out<T>(p.o) + b * p.so.b + h * p.so.h + t * p.so.t + col, p.scale * (decay * so + sd * u));
#pragma unroll
      for (int i = 0; i < RPT; ++i) S[i] = decay * S[i] + kk[i] * u;
      phase ^= 1;   // the other buffer: this one may still be read
    }
    if (!later) break;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) *repoint<floatx4>(Sp + (int64_t)i * p.dv) = S[i];
}

template <typename T, int DK>
hipError_t launch_dk(const GdrStepParams& p, hipStream_t s) {
  const int64_t units = p.B * p.Hv;
  // 32 columns a workgroup always: the most workgroups (few rows need them, many do not mind)
  const unsigned grid = (unsigned)(units * (p.dv / 32));
  hipLaunchKernelGGL((gdr_step_kernel<T, DK, 32>), dim3(grid), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const GdrStepParams& p, hipStream_t s) {
  switch (p.dk) {
    case 32: return launch_dk<T, 32>(p, s);
    case 64: return launch_dk<T, 64>(p, s);
    default: return launch_dk<T, 128>(p, s);
  }
}

}  // namespace

hipError_t launch_gdr_step(const GdrStepParams& p, hipStream_t s) {
  return p.dtype == KDA_DTYPE_BF16 ? launch_t<uint16_t>(p, s) : launch_t<float>(p, s);
}

}  // namespace kda
