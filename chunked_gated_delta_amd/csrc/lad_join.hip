// What stands between and behind the walks of linear attention with a decay for each head: the chain over the
// segments' states, the log-decay's gradient, and the sum over value heads that share a query/key head.
#include "lad_internal.h"

namespace kda {

namespace {

// S entering segment i + 1 = e^{decay of i} S entering i + segment i's own state, and its adjoint from the last segment
// down; in place.  Every thread holds 4 values of a state and asks for 8 segments at a time; bound by HBM
// (512 states of 64 KiB: 15.5 us, 4.4 TB/s), or by the trips to memory of the longest sequence (9 packed prompts: 13.4 us).
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

// The log-decay's gradient is a sum over pairs of tokens, dg_t = sum of c_ij over i >= t > j.  With the dots d_i = q_i . dq_i
// = sum of c_ij over j <= i and e_j = k_j . dk_j = sum over i >= j, their parts d', e' across chunks, and A_c the sum over the
// pairs with j before chunk c and i behind it,
//     dg_t = A_c + sum over t' >= t of the chunk (d - (e - e')) + sum over t' < t of the chunk e'
// where a chunk's own pairs cancel as the values that they are.  A_c = B_{c+1} - sum of the chunk's e' = B_c - sum of its
// d' with B_c, the sum over the pairs on both sides of the chunk's start, = <S, R> there.  B is known at both ends of a segment;
// the chunks are walked from the end where it is smaller, since its rounding goes with them to where everything may be small
// (a state that the first tokens forget).  A segment of one chunk has A = e^{decay} <S entering, R from behind>, without any
// difference; A is 0 where nothing enters or nothing lies behind.  exact: dw is a result in fp32; otherwise the walk is from
// the last chunk down.  All in double; a wavefront takes a chunk.  Bound by the states' trip from memory (2 x 4096 tokens, 160
// segments of 128 x 128: 12.7 us).
template <typename T>
__global__ __launch_bounds__(256) void lad_decay_grad_kernel(LadDecayGrad p) {
  __shared__ double part[2][4];
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63;
  const int64_t slot = blockIdx.x / (uint32_t)p.Hv;
  const int h = (int)(blockIdx.x % (uint32_t)p.Hv);
  LadSeg sg;
  if (!lad_find(p.seq_start, p.T, p.L, p.n_seq, slot, &sg)) {
    if (p.w_per_head && tid == 0) p.partial[slot * p.Hv + h] = 0.0;
    return;
  }
  const int64_t first = sg.seg * p.L, len = sg.len - first < p.L ? sg.len - first : p.L;
  const int64_t n_chunks = (len + kGdrChunk - 1) / kGdrChunk;
  const auto wave_sum = [](double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
  };
  const auto block_sum = [&](double x, double (&at)[4]) {
    x = wave_sum(x);
    if (lane == 0) at[wave] = x;
    __syncthreads();
    return at[0] + at[1] + at[2] + at[3];
  };
  const auto product = [&](const float* a, const float* b) {   // this thread's part
    double dot = 0.0;
    if (a && b)
#pragma unroll 8   // eight trips to memory at once
      for (int i = 4 * tid; i < p.size; i += 1024) {
        const floatx4 x = ld4f(global_in<float>(a) + i), y = ld4f(global_in<float>(b) + i);
#pragma unroll
        for (int r = 0; r < 4; ++r) dot += (double)x[r] * (double)y[r];
      }
    return dot;
  };
  // states at the segment's ends: of the chain, or as the call has them
  const bool chained = p.T > p.L, opens = sg.seg == 0, closes = sg.seg == sg.n_seg - 1;
  const auto of_slot = [&](const float* t, int64_t i) { return t + ((slot + i) * p.Hv + h) * p.size; };
  const auto of_seq = [&](const float* t) { return t ? t + (sg.seq * p.Hv + h) * p.size : nullptr; };
  const float *S_in = chained ? of_slot(p.s, 0) : of_seq(p.S0), *R_out = chained ? of_slot(p.r, 0) : of_seq(p.dSf);
  const float* S_out = closes ? (p.dSf ? of_seq(p.S_final) : nullptr) : of_slot(p.s, 1);
  const float* R_in = opens ? of_seq(p.dS0) : of_slot(p.r, -1);
  const bool one = p.exact && n_chunks == 1;
  bool down = true;
  double B;     // the sum at the end that the walk starts from
  if (one) {
    double g = 0.0;
    if (wave == 0 && lane < len)
      g = lad_decay<T>(p.w, p.w_per_head, p.sw, sg.row, h, sg.t0 + first + lane, p.gate, p.g_min);
    const double dot = block_sum(product(S_in, R_out), part[0]), total = block_sum(g, part[1]);
    B = S_in && R_out ? exp(total) * dot : 0.0;
  } else {
    B = block_sum(product(S_out, R_out), part[0]);
    if (p.exact && (!S_in || R_in)) {   // what enters is there, or nothing enters
      const double at_start = block_sum(product(S_in, R_in), part[1]);
      if (fabs(at_start) < fabs(B)) {
        down = false;
        B = at_start;
      }
    }
  }
  const int64_t at = (sg.row * p.Hv + h) * p.T + sg.t0 + first;
  double total = 0.0;
  for (int64_t done = 0; done < n_chunks; done += 4) {
    const int64_t c = down ? n_chunks - 1 - done - wave : done + wave, t = kGdrChunk * c + lane;
    const bool live = c >= 0 && t < len;
    double d_in = 0.0, e_in = 0.0, own = 0.0;
    if (live) {
      d_in = p.qdq[0][at + t];
      e_in = p.kdk[0][at + t];
      own = p.qdq[1][at + t] - (p.kdk[1][at + t] - e_in);
    }
    double before = e_in;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double more = __shfl_down(own, d), less = __shfl_up(before, d);
      if (lane + d < 64) own += more;
      if (lane >= d) before += less;
    }
    const double e_sum = __shfl(before, 63), d_sum = wave_sum(d_in);
    before -= e_in;
    __syncthreads();   // the values of the turn before have been read
    if (lane == 0) part[0][wave] = down ? d_sum - e_sum : e_sum - d_sum;
    __syncthreads();
    double mine = B;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < wave) mine += part[0][w];
      B += part[0][w];
    }
    if (!one) mine -= down ? e_sum : d_sum;
    if ((c == 0 && opens && !p.S0) || (c == n_chunks - 1 && closes && !p.dSf)) mine = 0.0;   // nothing enters, or nothing is behind
    if (!live) continue;
    const double dg = mine + own + before;
    if (p.w_per_head) total += dg;
    else {
      const int64_t tok = sg.t0 + first + t;
      const float w = get(global_in<T>(p.w) + sg.row * p.sw.b + h * p.sw.h + tok * p.sw.t);
      put(global_out<T>(p.dw) + sg.row * p.sdw.b + h * p.sdw.h + tok * p.sdw.t, (float)(dg * (double)gdr_gate_grad(w, p.gate, p.g_min)));
    }
  }
  if (!p.w_per_head) return;
  __syncthreads();
  total = block_sum(total, part[1]);
  if (tid == 0) p.partial[slot * p.Hv + h] = total;
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
