// The norms around a block and their gradients, one pass over each row:
//   n = x / rms(x) * weight      h = n * act(z)      s = residual + alpha h      y = s / rms(s) * next_weight
// with rms(t) = sqrt(mean(t^2) + eps); the norm of x, the gate, the residual and the norm of s may each be
// absent.  Bound by HBM: every tensor is read or written once.  NT threads hold a row in registers, in
// fp32, 8 consecutive values a vector access where the row allows it and strided single values otherwise;
// s is normalised before it is rounded.  8191 rows of 4096 in bf16 with both norms, the gate and the residual: 335 MB
// in 78 us, 4.3 TB/s (a large copy: 4.8); with 512 threads a row 81 us.
//
// The backward recomputes the row's forward from the same inputs (it reads the residual in place of s: as
// many bytes, and exact), and sums the weights' gradients over the rows a workgroup takes, in registers;
// the workgroups' sums are added up by a second kernel in a fixed order.  Each workgroup more is one more row for that
// kernel: 512 of them, two a compute unit.  131072 gated rows of 128 in bf16: 168 MB in 50 + 5 us; both norms, gate and
// residual, bf16: 8192 rows of 4096 (537 MB) 238 + 8 us, 4096 of 8192 288 + 13.  Rows of more than 4096 values with both norms do
// not fit 256 registers: 16 are spilled up to 8192 values, 284 to 306 above, and on the path of single values (an odd
// size or alignment) 128 to 132 and 625 to 629, so 4096 rows of 8191 take 918 + 16 us.  One norm above 8192 values spills 4 to 6, or
// 128 on the path of single values.
#include "gdr_internal.h"

namespace kda {

namespace {

constexpr int kMaxBwdBlocks = 512;

template <int NT>
__device__ __forceinline__ float row_sum(float x, float* lds, int group) {
  if constexpr (NT <= 64) {
#pragma unroll
    for (int d = 1; d < NT; d <<= 1) x += __shfl_xor(x, d);
    return x;
  } else {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) s += lds[w];
    return s;
  }
}

// values (v, 0..7) of this thread's part of a row of D values
template <int NT, bool VEC>
struct RowMap {
  int t, D;
  __device__ __forceinline__ int at(int v, int j) const { return VEC ? (v * NT + t) * 8 + j : (v * 8 + j) * NT + t; }
  __device__ __forceinline__ bool has(int v, int j) const { return at(v, VEC ? 0 : j) < D; }
};

template <typename T, int NT, int VPT, bool VEC>
__device__ __forceinline__ void load_part(GlobalPtr<const T> row, RowMap<NT, VEC> m, float (&x)[VPT * 8]) {
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if constexpr (VEC) {
      if (m.has(v, 0)) {
        const auto f = load_row8(row + m.at(v, 0));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v * 8 + j] = (float)f[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v * 8 + j] = 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v * 8 + j] = m.has(v, j) ? get(row + m.at(v, j)) : 0.f;
    }
  }
}

template <typename T, int NT, int VPT, bool VEC>
__device__ __forceinline__ void store_part(GlobalPtr<T> row, RowMap<NT, VEC> m, const float (&x)[VPT * 8]) {
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if constexpr (VEC) {
      if (m.has(v, 0)) {
        store_row4(row + m.at(v, 0), floatx4{x[v * 8], x[v * 8 + 1], x[v * 8 + 2], x[v * 8 + 3]});
        store_row4(row + m.at(v, 4), floatx4{x[v * 8 + 4], x[v * 8 + 5], x[v * 8 + 6], x[v * 8 + 7]});
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (m.has(v, j)) put(row + m.at(v, j), x[v * 8 + j]);
    }
  }
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// The place of row number (b H + h) T + t; the rows are fewer than 2^27 (checked on the host), so 32 bits divide
// them: a lane's two 64-bit divisions would be more instructions than the rest of a short row takes.
struct RowAt {
  uint32_t b, h, t;
  __device__ __forceinline__ RowAt(const NormParams& p, uint32_t row) {
    const uint32_t T = (uint32_t)p.T, H = (uint32_t)p.H, bh = row / T;
    t = row - bh * T;
    b = bh / H;
    h = bh - b * H;
  }
};
template <typename T> __device__ __forceinline__ GlobalPtr<T> row_of(const void* p, kda_stride_t s, const RowAt& i) {
  return (GlobalPtr<T>)p + i.b * s.b + i.h * s.h + i.t * s.t;
}

// the weight of this thread's values, in either type
template <typename T, int NT, int VPT, bool VEC>
__device__ __forceinline__ void load_weight(const void* w, int wdtype, RowMap<NT, VEC> m, float (&x)[VPT * 8]) {
  if (wdtype == KDA_DTYPE_BF16) load_part<uint16_t, NT, VPT, VEC>(global_in<uint16_t>(w), m, x);
  else load_part<float, NT, VPT, VEC>(global_in<float>(w), m, x);
}

template <typename T, int NT, int VPT, bool VEC, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_fwd_kernel(NormParams p) {
  constexpr int E = VPT * 8, GROUPS = THREADS / NT;
  __shared__ float lds[THREADS / 64];
  const int64_t rows = p.B * p.H * p.T;
  const int group = threadIdx.x / NT;
  const RowMap<NT, VEC> m{(int)(threadIdx.x % NT), (int)p.D};
  const int64_t row = (int64_t)blockIdx.x * GROUPS + group;
  if (row >= rows) return;
  const RowAt at(p, (uint32_t)row);
  float x[E], a[E], w[E];
  load_part<T, NT, VPT, VEC>(row_of<T>(p.x, p.sx, at), m, x);
  if (p.z) load_part<T, NT, VPT, VEC>(row_of<T>(p.z, p.sz, at), m, a);
  if (p.weight) {
    load_weight<T, NT, VPT, VEC>(p.weight, p.wdtype, m, w);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) q += x[e] * x[e];
    const float r = rsqrtf(row_sum<NT>(q, lds, group) / (float)p.D + p.eps);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= r * w[e];
  }
  if (p.z) {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= sigmoid(a[e]) * (p.act == KDA_ACT_SILU ? a[e] : 1.f);
  }
  if (p.res) {
    load_part<T, NT, VPT, VEC>(row_of<T>(p.res, p.sr, at), m, a);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = p.alpha * x[e] + a[e];
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= p.alpha;
  }
  store_part<T, NT, VPT, VEC>(row_of<T>(p.s, p.ss, at), m, x);
  if (p.weight2) {
    load_weight<T, NT, VPT, VEC>(p.weight2, p.wdtype, m, w);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) q += x[e] * x[e];
    const float r = rsqrtf(row_sum<NT>(q, lds, group) / (float)p.D + p.eps);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= r * w[e];
    store_part<T, NT, VPT, VEC>(row_of<T>(p.y, p.sy, at), m, x);
  }
}

// SECOND: with the norm of s.  Without it the kernel needs half the registers, so twice the rows are under way.
template <typename T, int NT, int VPT, bool VEC, int THREADS, bool SECOND>
__global__ __launch_bounds__(THREADS) void norm_bwd_kernel(NormParams p) {
  constexpr int E = VPT * 8, GROUPS = THREADS / NT;
  __shared__ float lds[THREADS / 64];
  __shared__ float acc[GROUPS > 1 ? GROUPS * NT * E : 1];
  const int64_t rows = p.B * p.H * p.T;
  const int group = threadIdx.x / NT;
  const RowMap<NT, VEC> m{(int)(threadIdx.x % NT), (int)p.D};
  float dw[E], dw2[SECOND ? E : 1], kept[VPT == 1 ? E : 1];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    dw[e] = 0.f;
    if constexpr (SECOND) dw2[e] = 0.f;
  }
  if constexpr (VPT == 1) {   // longer parts of a row leave no registers for it
    if (p.weight) load_weight<T, NT, VPT, VEC>(p.weight, p.wdtype, m, kept);
  }

  // every thread of a workgroup makes the same number of turns (the row sums hold barriers)
  for (int64_t first = (int64_t)blockIdx.x * GROUPS; first < rows; first += (int64_t)gridDim.x * GROUPS) {
    const bool live = first + group < rows;
    const int64_t row = live ? first + group : rows - 1;
    const RowAt at(p, (uint32_t)row);
    float x[E], n[E], a[E], g[E], w[E];
    load_part<T, NT, VPT, VEC>(row_of<T>(p.x, p.sx, at), m, x);
    if (p.ds) load_part<T, NT, VPT, VEC>(row_of<T>(p.ds, p.sds, at), m, g);
    else {
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = 0.f;
    }
    if (p.z) load_part<T, NT, VPT, VEC>(row_of<T>(p.z, p.sz, at), m, a);
    float r = 1.f;
    if (p.weight) {
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) q += x[e] * x[e];
      r = rsqrtf(row_sum<NT>(q, lds, group) / (float)p.D + p.eps);
    }
    if (p.weight) {
      if constexpr (VPT > 1) load_weight<T, NT, VPT, VEC>(p.weight, p.wdtype, m, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if constexpr (VPT == 1) w[e] = kept[e];
        x[e] *= r;            // x / rms(x)
        n[e] = x[e] * w[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) n[e] = x[e];
    }
    if constexpr (SECOND) {   // through the second norm: g becomes the whole gradient of s
      float s[E], res[E], dy[E], w2[E];
      if (p.res) load_part<T, NT, VPT, VEC>(row_of<T>(p.res, p.sr, at), m, res);
      load_part<T, NT, VPT, VEC>(row_of<T>(p.dy, p.sdy, at), m, dy);
      load_weight<T, NT, VPT, VEC>(p.weight2, p.wdtype, m, w2);
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s[e] = p.alpha * n[e];
        if (p.z) s[e] *= sigmoid(a[e]) * (p.act == KDA_ACT_SILU ? a[e] : 1.f);
        if (p.res) s[e] += res[e];
        q += s[e] * s[e];
      }
      const float r2 = rsqrtf(row_sum<NT>(q, lds, group) / (float)p.D + p.eps);
      float c = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s[e] *= r2;
        if (live) dw2[e] += dy[e] * s[e];
        dy[e] *= w2[e];
        c += dy[e] * s[e];
      }
      c = row_sum<NT>(c, lds, group) / (float)p.D;
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] += r2 * (dy[e] - s[e] * c);
    }
    if (p.dres && live) store_part<T, NT, VPT, VEC>(row_of<T>(p.dres, p.sdr, at), m, g);
#pragma unroll
    for (int e = 0; e < E; ++e) g[e] *= p.alpha;
    if (p.z) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float sg = sigmoid(a[e]);
        const float der = p.act == KDA_ACT_SILU ? sg * (1.f + a[e] * (1.f - sg)) : sg * (1.f - sg);
        const float val = p.act == KDA_ACT_SILU ? sg * a[e] : sg;
        a[e] = g[e] * n[e] * der;
        g[e] *= val;
      }
      if (p.dz && live) store_part<T, NT, VPT, VEC>(row_of<T>(p.dz, p.sdz, at), m, a);
    }
    if (p.weight) {
      float c = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (live) dw[e] += g[e] * x[e];
        g[e] *= w[e];
        c += g[e] * x[e];
      }
      c = row_sum<NT>(c, lds, group) / (float)p.D;
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = r * (g[e] - x[e] * c);
    }
    if (live) store_part<T, NT, VPT, VEC>(row_of<T>(p.dx, p.sdx, at), m, g);
  }

  // this workgroup's sums: the row groups' one after another
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !p.dweight : !p.dweight2) continue;
    const auto out = as_global(p.partial) + ((int64_t)which * kMaxBwdBlocks + blockIdx.x) * p.D;
    float d[E];
#pragma unroll
    for (int e = 0; e < E; ++e) d[e] = which == 0 ? dw[e] : dw2[SECOND ? e : 0];
    if constexpr (GROUPS > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) acc[(group * E + e) * NT + m.t] = d[e];
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float sum = 0.f;
#pragma unroll 2   // whole, it would take more registers than the rows
          for (int q = 0; q < GROUPS; ++q) sum += acc[(q * E + e) * NT + m.t];
          d[e] = sum;
        }
      }
    }
    if (group == 0) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (m.at(v, j) < p.D) out[m.at(v, j)] = d[v * 8 + j];
    }
  }
}

// adds up the workgroups' sums: 16 columns a workgroup, 64 threads along the workgroups of each
__global__ __launch_bounds__(1024) void norm_weight_kernel(NormParams p, int blocks) {
  __shared__ float part[64][17];
  const int c = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + c;
  const int which = blockIdx.y;
  void* out = which == 0 ? p.dweight : p.dweight2;
  if (!out) return;
  const auto in = global_in<float>(p.partial) + (int64_t)which * kMaxBwdBlocks * p.D;
  float s = 0.f;
  if (col < p.D) {
    int i = y;
    for (; i + 7 * 64 < blocks; i += 8 * 64) {   // eight loads under way at once
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = in[(int64_t)(i + 64 * k) * p.D + col];
#pragma unroll
      for (int k = 0; k < 8; ++k) s += x[k];
    }
    for (; i < blocks; i += 64) s += in[(int64_t)i * p.D + col];
  }
  part[y][c] = s;
  __syncthreads();
  if (y == 0 && col < p.D) {
    s = 0.f;
    for (int i = 0; i < 64; ++i) s += part[i][c];
    if (p.wdtype == KDA_DTYPE_BF16) put(global_out<uint16_t>(out) + col, s);
    else put(global_out<float>(out) + col, s);
  }
}

bool vec_ok(const void* ptr, kda_stride_t s, int esz) {
  if (!ptr) return true;
  const int64_t per = 16 / esz;
  return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0 && s.b % per == 0 && s.h % per == 0 && s.t % per == 0;
}

template <typename T, int NT, int VPT, bool VEC>
hipError_t launch_one(const NormParams& p, hipStream_t s, bool bwd) {
  const int64_t rows = p.B * p.H * p.T;
  if (!bwd) {
    constexpr int THREADS = NT > 256 ? NT : 256, GROUPS = THREADS / NT;
    hipLaunchKernelGGL((norm_fwd_kernel<T, NT, VPT, VEC, THREADS>), dim3((unsigned)((rows + GROUPS - 1) / GROUPS)), dim3(THREADS), 0, s, p);
    return hipGetLastError();
  }
  // Short rows: workgroups of 8 wavefronts, so that two a compute unit put 16 rows' loads more under way (gradients
  // of 131072 gated rows of 128: 50 us against 55 with 4 wavefronts and 58 with 16); 16 values a lane have no
  // registers for that.
  constexpr int THREADS = NT > 256 || (NT <= 64 && VPT == 1) ? 512 : 256, GROUPS = THREADS / NT;
  const int64_t blocks = (rows + GROUPS - 1) / GROUPS;
  const int grid = (int)(blocks < kMaxBwdBlocks ? blocks : kMaxBwdBlocks);
  if (grid == 0) {}   // no rows: the weights' sums alone
  else if (p.weight2) hipLaunchKernelGGL((norm_bwd_kernel<T, NT, VPT, VEC, THREADS, true>), dim3(grid), dim3(THREADS), 0, s, p);
  else hipLaunchKernelGGL((norm_bwd_kernel<T, NT, VPT, VEC, THREADS, false>), dim3(grid), dim3(THREADS), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.dweight && !p.dweight2)) return e;
  hipLaunchKernelGGL(norm_weight_kernel, dim3((unsigned)((p.D + 15) / 16), 2), dim3(1024), 0, s, p, grid);
  return hipGetLastError();
}

// threads along a row: 8 values each, up to 32
template <typename T, bool VEC>
hipError_t launch_d(const NormParams& p, hipStream_t s, bool bwd) {
  if (p.D <= 128) return launch_one<T, 16, 1, VEC>(p, s, bwd);
  if (p.D <= 512) return launch_one<T, 64, 1, VEC>(p, s, bwd);
  if (p.D <= 1024) return launch_one<T, 64, 2, VEC>(p, s, bwd);
  if (p.D <= 2048) return launch_one<T, 256, 1, VEC>(p, s, bwd);
  if (p.D <= 4096) return launch_one<T, 256, 2, VEC>(p, s, bwd);
  if (p.D <= 8192) return launch_one<T, 512, 2, VEC>(p, s, bwd);
  return launch_one<T, 512, 4, VEC>(p, s, bwd);
}

hipError_t launch_norm(const NormParams& p, hipStream_t s, bool bwd) {
  const int esz = p.dtype == KDA_DTYPE_BF16 ? 2 : 4;
  const kda_stride_t zero = {0, 0, 0};
  const bool vec = p.D % 8 == 0 && vec_ok(p.x, p.sx, esz) && vec_ok(p.z, p.sz, esz) && vec_ok(p.res, p.sr, esz) &&
                   vec_ok(p.s, p.ss, esz) && vec_ok(p.y, p.sy, esz) && vec_ok(p.ds, p.sds, esz) && vec_ok(p.dy, p.sdy, esz) &&
                   vec_ok(p.dx, p.sdx, esz) && vec_ok(p.dz, p.sdz, esz) && vec_ok(p.dres, p.sdr, esz) &&
                   vec_ok(p.weight, zero, esz) && vec_ok(p.weight2, zero, esz);
  if (p.dtype == KDA_DTYPE_BF16) return vec ? launch_d<uint16_t, true>(p, s, bwd) : launch_d<uint16_t, false>(p, s, bwd);
  return vec ? launch_d<float, true>(p, s, bwd) : launch_d<float, false>(p, s, bwd);
}

}  // namespace

size_t norm_bwd_workspace_bytes(const NormParams& p) { return (size_t)2 * kMaxBwdBlocks * p.D * 4; }
hipError_t launch_norm_fwd(const NormParams& p, hipStream_t s) { return launch_norm(p, s, false); }
hipError_t launch_norm_bwd(const NormParams& p, hipStream_t s) { return launch_norm(p, s, true); }

}  // namespace kda
