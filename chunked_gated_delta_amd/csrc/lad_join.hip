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
// where a chunk's own pairs cancel as the values that they are.  With B_c, the sum over the pairs on both sides of the
// chunk's start, A_c = B_c - sum of its d' = B_{c+1} - sum of its e'.  B = <S, R> is known at both ends of a segment (0 where
// nothing enters or nothing lies behind), so A is carried from either end.  Every sum that goes into it leaves its rounding
// there, also where the head has forgotten what made it large, so each chunk takes the end whose values on the way were smaller.
// And A_c has the chunk's whole decay as a factor: where 0 is nearer to it than the rounding of what is carried (a
// reset, a decay of more than a half a token), it is 0 and both ways start anew; unless what is carried stands out of its rounding
// (masked tokens between two states: <S, R> is all there is).  Between a part that forgets and one that remembers
// (2048 tokens, decays of 2 and 1/2048 a token, fp32) the first one's gradients were off by 1.7e-3 where A came from the far end.
// A segment of one chunk has A = e^{decay} <S entering, R from behind>, without any difference.  All in double; a wavefront
// takes a chunk.  Bound by the states' trip from memory (2 x 4096 tokens, 160 segments of 128 x 128, four states each: 12.9 us).
template <typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void lad_decay_grad_kernel(LadDecayGrad p) {
  extern __shared__ __attribute__((aligned(16))) char raw[];
  __shared__ double part[4][WAVES];
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63;
  const int64_t slot = blockIdx.x / (uint32_t)p.Hv;
  const int h = (int)(blockIdx.x % (uint32_t)p.Hv);
  LadSeg sg;
  if (!lad_find(p.seq_start, p.T, p.L, p.n_seq, slot, &sg)) {
    if (p.w_per_head && tid == 0) p.partial[slot * p.Hv + h] = 0.0;
    return;
  }
  const int64_t first = sg.seg * p.L, len = sg.len - first < p.L ? sg.len - first : p.L;
  const int n_chunks = (int)((len + kGdrChunk - 1) / kGdrChunk), most = (int)(p.L / kGdrChunk);
  // by chunk: sums of d' and e' and their sizes, e^{decay}; A from the start and from the end, and the size of what it was taken from
  double* const d_sum = reinterpret_cast<double*>(raw);
  double *const e_sum = d_sum + most, *const A_up = e_sum + most, *const A_down = A_up + most;
  float* const d_size = reinterpret_cast<float*>(A_down + most);
  float *const e_size = d_size + most, *const kept = e_size + most, *const size_up = kept + most, *const size_down = size_up + most;
  const int64_t at = (sg.row * p.Hv + h) * p.T + sg.t0 + first;
  // states at the segment's ends: of the chain, or as the call has them
  const bool chained = p.T > p.L, opens = sg.seg == 0, closes = sg.seg == sg.n_seg - 1;
  const auto of_slot = [&](const float* t, int64_t i) { return t + ((slot + i) * p.Hv + h) * p.size; };
  const auto of_seq = [&](const float* t) { return t ? t + (sg.seq * p.Hv + h) * p.size : nullptr; };
  const float *S_in = chained ? of_slot(p.s, 0) : of_seq(p.S0), *R_out = chained ? of_slot(p.r, 0) : of_seq(p.dSf);
  const float *S_out = closes ? (p.dSf ? of_seq(p.S_final) : nullptr) : of_slot(p.s, 1);
  const float *R_in = opens ? (p.S0 ? of_seq(p.dS0) : nullptr) : of_slot(p.r, -1);
  // their product, and the size of its terms, as sums of the wavefronts' parts
  const auto product = [&](const float* a, const float* b, double* sum, double* size) {
    double dot = 0.0, sq = 0.0;
    if (a && b)
#pragma unroll 4   // eight trips to memory at once
      for (int i = 4 * tid; i < p.size; i += 256 * WAVES) {
        const floatx4 x = ld4f(global_in<float>(a) + i), y = ld4f(global_in<float>(b) + i);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const double term = (double)x[r] * (double)y[r];
          dot += term;
          sq += term * term;
        }
      }
    dot = lane_sum(dot);
    sq = lane_sum(sq);
    if (lane == 0) {
      sum[wave] = dot;
      size[wave] = sq;
    }
  };
  const auto all = [](const double* x) {
    double s = 0.0;
    for (int w = 0; w < WAVES; ++w) s += x[w];
    return s;
  };
  // a wavefront's first chunk is on its way beside the states
  double d, e;
  float g;
  const auto ask = [&](int c) {
    const int64_t t = kGdrChunk * (int64_t)c + lane;
    const bool live = t < len;
    d = live ? p.qdq[0][at + t] : 0.0;
    e = live ? p.kdk[0][at + t] : 0.0;
    g = live ? lad_decay<T>(p.w, p.w_per_head, p.sw, sg.row, h, sg.t0 + first + t, p.gate, p.g_min) : 0.f;
  };
  ask(wave);
  if (n_chunks == 1) product(S_in, R_out, part[0], part[1]);
  else if (n_chunks > 1) {
    product(S_in, R_in, part[0], part[1]);
    product(S_out, R_out, part[2], part[3]);
  }
  for (int c = wave; c < n_chunks; c += WAVES) {
    if (c != wave) ask(c);
    const double ds = lane_sum(d), es = lane_sum(e), decay = lane_sum((double)g);
    const float dn = lane_sum((float)fabs(d)), en = lane_sum((float)fabs(e));
    if (lane == 0) {
      d_sum[c] = ds;
      e_sum[c] = es;
      d_size[c] = 0.125f * dn;   // of 64 values with signs of their own
      e_size[c] = 0.125f * en;
      kept[c] = (float)exp(decay);
      if (n_chunks == 1) A_up[0] = exp(decay);
    }
  }
  __syncthreads();
  if (n_chunks == 1) {
    if (tid == 0) {
      A_up[0] = S_in && R_out ? A_up[0] * all(part[0]) : 0.0;
      size_up[0] = size_down[0] = 0.f;
    }
  } else if (n_chunks > 1) {
    if (lane == 0 && wave < 2) {
      const bool down = wave == 1;
      const float ends[2] = {(float)sqrt(all(part[1])), (float)sqrt(all(part[3]))};
      float whole = ends[0] + ends[1];
      for (int c = 0; c < n_chunks; ++c) whole += d_size[c] + e_size[c];
      // A without its factor, a product of two states, is taken as at most 2^20 times the values' size; their rounding is 2^-22 of it
      const float far = 0x1p42f * whole;
      const double *const near_sum = down ? e_sum : d_sum, *const far_sum = down ? d_sum : e_sum;
      const float *const near_size = down ? e_size : d_size, *const far_size = down ? d_size : e_size;
      double* const A_out = down ? A_down : A_up;
      float* const size_out = down ? size_down : size_up;
      double B = all(down ? part[2] : part[0]);
      float size = ends[down];
      for (int i = 0; i < n_chunks; ++i) {
        const int c = down ? n_chunks - 1 - i : i;
        double A = B - near_sum[c];
        size += near_size[c];
        const float to_zero = kept[c] == 0.f ? 0.f : kept[c] * far;
        if (to_zero < size && fabs(A) <= 0x1p-12 * (double)size) {   // and what is carried does not say that it is more
          A = 0.0;
          size = to_zero;
        }
        A_out[c] = A;
        size_out[c] = size;
        B = A + far_sum[c];
        size += far_size[c];
      }
    }
  }
  __syncthreads();
  double total = 0.0;
  for (int c = wave; c < n_chunks; c += WAVES) {
    const int64_t t = kGdrChunk * (int64_t)c + lane;
    const bool live = t < len;
    double e_in = 0.0, own = 0.0;
    if (live) {
      e_in = p.kdk[0][at + t];
      own = p.qdq[1][at + t] - (p.kdk[1][at + t] - e_in);
    }
    const double before = lane_prefix(e_in) - e_in, upto = lane_prefix(own);
    own += last_lane(upto) - upto;   // from this token on
    if (!live) continue;
    const double dg = (size_down[c] < size_up[c] ? A_down[c] : A_up[c]) + own + before;
    if (p.w_per_head) total += dg;
    else {
      const int64_t tok = sg.t0 + first + t;
      const float w = get(global_in<T>(p.w) + sg.row * p.sw.b + h * p.sw.h + tok * p.sw.t);
      put(global_out<T>(p.dw) + sg.row * p.sdw.b + h * p.sdw.h + tok * p.sdw.t, (float)(dg * (double)gdr_gate_grad(w, p.gate, p.g_min)));
    }
  }
  if (!p.w_per_head) return;
  total = lane_sum(total);
  if (lane == 0) part[0][wave] = total;
  __syncthreads();
  if (tid == 0) p.partial[slot * p.Hv + h] = all(part[0]);
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
  const unsigned lds = (unsigned)(p.L / kGdrChunk) * (4 * sizeof(double) + 5 * sizeof(float));   // at most kLadMaxChunks: 52 KiB
  // Few workgroups wait for their states from memory, and 16 wavefronts have more of them under way than 4 (2 x 4096 tokens, 160 of
  // them: 25 and 16 us when this was chosen); many hide it behind one another, and wavefronts without a chunk of their own are in the way.
  if (p.slots * p.Hv <= 1024) {
    if (p.dtype == KDA_DTYPE_BF16) hipLaunchKernelGGL((lad_decay_grad_kernel<uint16_t, 16>), grid, dim3(1024), lds, s, p);
    else hipLaunchKernelGGL((lad_decay_grad_kernel<float, 16>), grid, dim3(1024), lds, s, p);
  } else {
    if (p.dtype == KDA_DTYPE_BF16) hipLaunchKernelGGL((lad_decay_grad_kernel<uint16_t, 4>), grid, dim3(256), lds, s, p);
    else hipLaunchKernelGGL((lad_decay_grad_kernel<float, 4>), grid, dim3(256), lds, s, p);
  }
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
