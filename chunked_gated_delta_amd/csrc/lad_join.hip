// What stands between and behind the walks of linear attention with a decay for each head: the chain over the
// segments' states, the log-decay's gradient, and the sum over value heads that share a query/key head.
#include "lad_internal.h"

namespace kda {

namespace {

// S entering segment i + 1 = e^{decay of i} S entering i + segment i's own state, and its adjoint from the last segment
// down; in place.  Every thread holds 4 values of a state and asks for 8 segments at a time; bound by HBM, or by
// the trips to memory of the longest sequence.
__global__ __launch_bounds__(256) void lad_scan_kernel(LadScan p) {
  const int per = (p.size + 1023) / 1024;
  const uint32_t unit = blockIdx.x / (uint32_t)per, dirs = (uint32_t)p.dirs;
  const int dir = (int)(unit % dirs), h = (int)(unit / dirs % (uint32_t)p.Hv);
  const int64_t seq = unit / dirs / (uint32_t)p.Hv;
  const int64_t at = (blockIdx.x % per) * 1024 + 4 * threadIdx.x;
  if (at >= p.size) return;
  const LadSeg sg = lad_seq(p.seq_start, p.T, p.L, seq);
  const auto base = as_global(dir ? p.r : p.s);
  const auto decay = global_in<float>(dir ? p.r_decay : p.s_decay);
  const float* in = dir ? p.dSf : p.S0;
  float* out = dir ? p.dS0 : p.S_final;
  const int64_t whole = (seq * p.Hv + h) * p.size + at;
  floatx4 x = {};
  if (in) x = ld4f(global_in<float>(in) + whole);
  const int64_t n = sg.n_seg;
  const auto slot = [&](int64_t i) { return (sg.slot0 + (dir ? n - 1 - i : i)) * p.Hv + h; };
  // the last one's own state counts only where something leaves it
  const int64_t own = out ? n : n - 1;
  for (int64_t i = 0; i < n; i += 8) {
    floatx4 add[8];
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t s = slot(i + j < own ? i + j : 0);
      const bool live = i + j < own;
      add[j] = live ? ld4f(base + s * p.size + at) : floatx4{};
      a[j] = live ? decay[s] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) {
        *repoint<floatx4>(base + slot(i + j) * p.size + at) = x;
        x = a[j] * x + add[j];
      }
  }
  if (out) *repoint<floatx4>(as_global(out) + whole) = x;
}

// The log-decay's gradient is a sum over pairs of tokens, dg_t = sum of c_ij over i >= t > j; with B_c the sum over the
// pairs on both sides of chunk c's start (= <S, R> there), and the dots d_i = q_i . dq_i = sum of c_ij over j <= i,
// e_j = k_j . dk_j = sum of c_ij over i >= j, each also without its chunk's own pairs (d', e'):
//     dg_t = B_{c+1} + sum over t' >= t of the chunk (d - e),   B_c = B_{c+1} + sum over the chunk (d' - e')
// A chunk's own pairs cancel in its d and e; left out of B they leave no rounding there, which would come from as many
// tokens as the segment has and be large beside the gradient of a head that soon forgets.  B at the segment's end is the product
// of states.  All in double; a wavefront takes a chunk, from the last one down.
template <typename T>
__global__ __launch_bounds__(256) void lad_decay_grad_kernel(LadDecayGrad p) {
  __shared__ double part[4];
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63;
  const int64_t slot = blockIdx.x / (uint32_t)p.Hv;
  const int h = (int)(blockIdx.x % (uint32_t)p.Hv);
  LadSeg sg;
  if (!lad_find(p.seq_start, p.T, p.L, p.n_seq, slot, &sg)) {
    if (p.w_per_head && tid == 0) p.partial[slot * p.Hv + h] = 0.0;
    return;
  }
  const int64_t first = sg.seg * p.L, len = sg.len - first < p.L ? sg.len - first : p.L;
  const auto wave_sum = [](double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
  };
  // <S, R> where the segment ends
  const bool last = sg.seg == sg.n_seg - 1;
  const float *S = nullptr, *R = nullptr;
  if (!last) {
    S = p.s + ((slot + 1) * p.Hv + h) * p.size;
    R = p.r + (slot * p.Hv + h) * p.size;
  } else if (p.dSf) {
    S = p.S_final + (sg.seq * p.Hv + h) * p.size;
    R = p.dSf + (sg.seq * p.Hv + h) * p.size;
  }
  double dot = 0.0;
  if (S)
#pragma unroll 8   // eight trips to memory at once
    for (int i = 4 * tid; i < p.size; i += 1024) {
      const floatx4 a = ld4f(global_in<float>(S) + i), b = ld4f(global_in<float>(R) + i);
#pragma unroll
      for (int r = 0; r < 4; ++r) dot += (double)a[r] * (double)b[r];
    }
  dot = wave_sum(dot);
  if (lane == 0) part[wave] = dot;
  __syncthreads();
  double B = part[0] + part[1] + part[2] + part[3];   // behind the chunks taken so far
  const int64_t at = (sg.row * p.Hv + h) * p.T + sg.t0 + first;
  const int64_t n_chunks = (len + kGdrChunk - 1) / kGdrChunk;
  double total = 0.0;
  for (int64_t done = 0; done < n_chunks; done += 4) {
    const int64_t c = n_chunks - 1 - done - wave, t = kGdrChunk * c + lane;
    const bool live = c >= 0 && t < len;
    double own = 0.0, across = 0.0;
    if (live) {
      own = p.qdq[1][at + t] - p.kdk[1][at + t];
      across = p.qdq[0][at + t] - p.kdk[0][at + t];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double more = __shfl_down(own, d);
      if (lane + d < 64) own += more;
    }
    across = wave_sum(across);
    __syncthreads();   // the values of the turn before have been read
    if (lane == 0) part[wave] = across;
    __syncthreads();
    double mine = B;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < wave) mine += part[w];
      B += part[w];
    }
    if (!live) continue;
    const double dg = mine + own;
    if (p.w_per_head) total += dg;
    else {
      const int64_t tok = sg.t0 + first + t;
      const float w = get(global_in<T>(p.w) + sg.row * p.sw.b + h * p.sw.h + tok * p.sw.t);
      put(global_out<T>(p.dw) + sg.row * p.sdw.b + h * p.sdw.h + tok * p.sdw.t, (float)(dg * (double)gdr_gate_grad(w, p.gate, p.g_min)));
    }
  }
  if (!p.w_per_head) return;
  total = wave_sum(total);
  __syncthreads();
  if (lane == 0) part[wave] = total;
  __syncthreads();
  if (tid == 0) p.partial[slot * p.Hv + h] = part[0] + part[1] + part[2] + part[3];
}

// dw of a w per head: the segments' sums, in a fixed order
__global__ __launch_bounds__(256) void lad_head_grad_kernel(LadDecayGrad p) {
  __shared__ double part[256];
  const int tid = threadIdx.x, h = blockIdx.x;
  double sum = 0.0;
  for (int64_t i = tid; i < p.slots; i += 256) sum += p.partial[i * p.Hv + h];
  part[tid] = sum;
  __syncthreads();
  for (int d = 128; d > 0; d >>= 1) {
    if (tid < d) part[tid] += part[tid + d];
    __syncthreads();
  }
  if (tid == 0) static_cast<float*>(p.dw)[h] = (float)(part[0] * (double)gdr_gate_grad(static_cast<const float*>(p.w)[h], p.gate, p.g_min));
}

template <typename T>
__global__ __launch_bounds__(256) void lad_sum_kernel(LadSum p) {
  const int per = p.D / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.B * p.Hk * p.T * per; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per, t = row % p.T, bh = row / p.T, b = bh / p.Hk;
    const int c = (int)(i % per) * 4, h = (int)(bh % p.Hk);
    if (p.seq_start && (t < p.seq_start[0] || t >= p.seq_start[p.n_seq])) continue;   // of no sequence
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      floatx4 x = {};
      for (int g = 0; g < p.grp; ++g) x += ld4f(global_in<float>(p.part[j]) + ((bh * p.grp + g) * p.T + t) * p.D + c);
      store_row4(global_out<T>(p.out[j]) + b * p.so[j].b + h * p.so[j].h + t * p.so[j].t + c, x);
    }
  }
}

}  // namespace

hipError_t launch_lad_scan(const LadScan& p, hipStream_t s) {
  const int64_t grid = p.n_seq * p.Hv * p.dirs * ((p.size + 1023) / 1024);
  hipLaunchKernelGGL(lad_scan_kernel, dim3((unsigned)grid), dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_lad_decay_grad(const LadDecayGrad& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.slots * p.Hv));
  if (p.dtype == KDA_DTYPE_BF16) hipLaunchKernelGGL(lad_decay_grad_kernel<uint16_t>, grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL(lad_decay_grad_kernel<float>, grid, dim3(256), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.w_per_head) return e;
  hipLaunchKernelGGL(lad_head_grad_kernel, dim3((unsigned)p.Hv), dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_lad_sum(const LadSum& p, hipStream_t s) {
  const int64_t n = p.B * p.Hk * p.T * (p.D / 4);
  const int64_t blocks = (n + 255) / 256, most = 1 << 20;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  if (p.dtype == KDA_DTYPE_BF16) hipLaunchKernelGGL(lad_sum_kernel<uint16_t>, grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL(lad_sum_kernel<float>, grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace kda
