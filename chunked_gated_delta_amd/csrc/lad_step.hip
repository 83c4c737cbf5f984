// Recurrent step of linear attention with a decay for each head on a pool of resident states, a few tokens a row.
//
// Bound by the state's two trips through HBM (512 rows of 16 heads, 128 x 128: 219 us, 4.9 TB/s; one row: 4.6 us).  A workgroup owns one (row, value head) and 32 value columns; a thread
// holds 4 columns (one 16-byte access) of DK / 32 consecutive state rows for all the call's tokens.  The new state
// needs no sum, and the output one over the state rows (lanes by shuffles, wavefronts through LDS):
//   S <- e^g S + k v^T,   o = scale S^T q
//
// Rows that name the same slot are successive tokens of that state: the first such row's workgroup takes them all
// in order and the others return, so no two workgroups touch one state.
#include "lad_internal.h"

namespace kda {

namespace {

template <typename T, int DK>
__global__ __launch_bounds__(256) void lad_step_kernel(LadStepParams p) {
  constexpr int CB = 32, CT = CB / 4;    // columns of a workgroup, threads along them
  constexpr int RG = 256 / CT;           // row groups
  constexpr int RPT = DK / RG;           // state rows of a thread
  static_assert(RPT >= 1, "tile");
  __shared__ __attribute__((aligned(16))) float part[2][4][CB];
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
      const float decay = expf(lad_decay<T>(p.w, p.w_per_head, p.sw, b, h, t, p.gate, p.g_min));
      floatx4 o = {};
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        S[i] = decay * S[i] + get(kp + i) * v;
        o += S[i] * get(qp + i);
      }
#pragma unroll
      for (int m = CT; m < 64; m <<= 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] += __shfl_xor(o[r], m);
      }
      if (lane < CT) *reinterpret_cast<floatx4*>(part[phase][wave] + 4 * ct) = o;
      block_barrier();
      if (rg == 0) {
        floatx4 s = {};
#pragma unroll
        for (int w = 0; w < 4; ++w) s += *reinterpret_cast<const floatx4*>(part[phase][w] + 4 * ct);
        store_row4(global_out<T>(p.o) + b * p.so.b + h * p.so.h + t * p.so.t + col, p.scale * s);
      }
      phase ^= 1;   // the other buffer: this one may still be read
    }
    if (!later) break;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) *repoint<floatx4>(Sp + (int64_t)i * p.dv) = S[i];
}

template <typename T>
hipError_t launch_t(const LadStepParams& p, hipStream_t s) {
  const unsigned grid = (unsigned)(p.B * p.Hv * (p.dv / 32));
  switch (p.dk) {
    case 32: hipLaunchKernelGGL((lad_step_kernel<T, 32>), dim3(grid), dim3(256), 0, s, p); break;
    case 64: hipLaunchKernelGGL((lad_step_kernel<T, 64>), dim3(grid), dim3(256), 0, s, p); break;
    default: hipLaunchKernelGGL((lad_step_kernel<T, 128>), dim3(grid), dim3(256), 0, s, p); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lad_step(const LadStepParams& p, hipStream_t s) {
  return p.dtype == KDA_DTYPE_BF16 ? launch_t<uint16_t>(p, s) : launch_t<float>(p, s);
}

}  // namespace kda
