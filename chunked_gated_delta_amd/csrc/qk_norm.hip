// Norms of queries and keys for each head with the rotation by position, and their gradients, one pass over each row:
//   n = x / rms(x) * weight,   y = scale * rot(n):  (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first R
// values.  Bound by HBM where there are many rows (16K tokens, 32 + 8 heads of 128 in bf16: 69 us, 4.9 TB/s; gradients of
// 8192 tokens, 16 + 16 heads: 39 us, 5.2 TB/s, and 4 us for the weights' sums), by the call where there are few.
//
// NT lanes hold a row as 8 pairs each; a group of NT lanes keeps one token and walks its heads, so the sines of a
// token's angles are formed once for all of them (64 pairs cost more than a row's trip through memory would).
// Angles are products of the position and the fp32 frequency in double, reduced to a turn there (a float's product is off
// by 0.03 radians at position 10^6) and rounded once to fp32 for the sine and cosine: off by at most 2^-25 of a half turn.
//
// The gradient recomputes the norm from the same row; the weights' gradients are summed in registers over the rows that a
// workgroup takes, and a second kernel adds up the workgroups in a fixed order.
#include "lad_internal.h"

namespace kda {

namespace {

constexpr int kMaxBlocks = 512;   // workgroups a tensor of the gradient: rows of partial sums

// How a lane's 8 pairs lie in a row.  kWhole: consecutive, moved in 16-byte pieces at whatever place they lie (this
// hardware's vector accesses need no more than the type's alignment); the pairs that turn and those that do not (one kind
// where they are neighbours) come in whole groups of 8.  kOver: the same, the last group of a kind reaching back over pairs
// of the one before, which both write alike and only the first counts; each kind has none or at least 8.  kSingle: pairs NT
// apart, one value at a time.
enum { kSingle, kWhole, kOver };
template <int NT, bool NEAR, int FORM> struct Pairs {
  int t, D, R;
  int a0, b0, twice, turn;   // first values of the run (a, b), pairs of it that count elsewhere, its first frequency
  bool live;                 // the lane has pairs
  __device__ __forceinline__ Pairs(int t_, int D_, int R_) : t(t_), D(D_), R(R_), a0(0), b0(0), twice(0), turn(0), live(true) {
    if constexpr (FORM != kSingle) {
      const int turning = NEAR ? D / 2 : R / 2, groups = (turning + 7) / 8;
      const bool turns = t < groups;
      const int kind = turns ? turning : D / 2 - turning, first = 8 * (turns ? t : t - groups);
      live = first < kind;
      const int s = !live ? 0 : FORM == kWhole || first + 8 <= kind ? first : kind - 8;
      twice = live ? first - s : 0;
      turn = turns || !live ? s : R / 2;
      a0 = NEAR ? 2 * s : turns || !live ? s : R + s;
      b0 = NEAR ? 2 * s + 1 : turns || !live ? s + R / 2 : R + s + kind;
    }
  }
  __device__ __forceinline__ bool has(int j) const { return FORM == kSingle ? j * NT + t < D / 2 : live; }
  __device__ __forceinline__ bool counts(int j) const { return FORM == kSingle ? j * NT + t < D / 2 : FORM == kWhole ? live : live && j >= twice; }
  __device__ __forceinline__ int frequency(int j) const { return FORM == kSingle ? j * NT + t : turn + j; }   // R / 2 and more: none
  // places of the pair's two values
  __device__ __forceinline__ int a(int j) const {
    if constexpr (FORM != kSingle) return a0 + (NEAR ? 2 * j : j);
    const int p = j * NT + t;
    return NEAR ? 2 * p : p < R / 2 ? p : R / 2 + p;
  }
  __device__ __forceinline__ int b(int j) const {
    if constexpr (FORM != kSingle) return b0 + (NEAR ? 2 * j : j);
    const int p = j * NT + t;
    return NEAR ? 2 * p + 1 : p < R / 2 ? p + R / 2 : p + D / 2;
  }
};

typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ bf16x8 load_any8(GlobalPtr<const uint16_t> p) { return __builtin_bit_cast(bf16x8, *repoint<u32x4_at2>(p)); }
__device__ __forceinline__ float8v load_any8(GlobalPtr<const float> p) {
  const floatx4 a = __builtin_bit_cast(floatx4, *repoint<u32x4_at4>(p)), b = __builtin_bit_cast(floatx4, *repoint<u32x4_at4>(p + 4));
  return float8v{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ float8v widen(bf16x8 f) { return __builtin_convertvector(__builtin_bit_cast(bf16x8v, f), float8v); }
__device__ __forceinline__ float8v widen(const float8v& f) { return f; }

template <typename T, int NT, bool NEAR, int FORM>
__device__ __forceinline__ void load_pairs(GlobalPtr<const T> row, const Pairs<NT, NEAR, FORM>& m, float (&a)[8], float (&b)[8]) {
  if constexpr (FORM != kSingle) {   // a lane without pairs reads the row's first values and drops them
    const float8v x = widen(load_any8(row + m.a0)), y = widen(load_any8(row + (NEAR ? m.a0 + 8 : m.b0)));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = NEAR ? (j < 4 ? x[2 * (j & 3)] : y[2 * (j & 3)]) : x[j];
      b[j] = NEAR ? (j < 4 ? x[2 * (j & 3) + 1] : y[2 * (j & 3) + 1]) : y[j];
      if (!m.live) a[j] = b[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = b[j] = 0.f;
      if (m.has(j)) {
        a[j] = get(row + m.a(j));
        b[j] = get(row + m.b(j));
      }
    }
  }
}

__device__ __forceinline__ void store8(GlobalPtr<uint16_t> p, const float (&x)[8]) {
  *repoint<u32x4_at2>(p) = u32x4_at2{pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7])};
}
__device__ __forceinline__ void store8(GlobalPtr<float> p, const float (&x)[8]) {
  *repoint<u32x4_at4>(p) = __builtin_bit_cast(u32x4_at4, floatx4{x[0], x[1], x[2], x[3]});
  *repoint<u32x4_at4>(p + 4) = __builtin_bit_cast(u32x4_at4, floatx4{x[4], x[5], x[6], x[7]});
}

template <typename T, int NT, bool NEAR, int FORM>
__device__ __forceinline__ void store_pairs(GlobalPtr<T> row, const Pairs<NT, NEAR, FORM>& m, const float (&a)[8], const float (&b)[8]) {
  if constexpr (FORM != kSingle) {
    if (!m.live) return;
    if constexpr (NEAR) {
      const float x[8] = {a[0], b[0], a[1], b[1], a[2], b[2], a[3], b[3]}, y[8] = {a[4], b[4], a[5], b[5], a[6], b[6], a[7], b[7]};
      store8(row + m.a0, x);
      store8(row + m.a0 + 8, y);
    } else {
      store8(row + m.a0, a);
      store8(row + m.b0, b);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (m.has(j)) {
        put(row + m.a(j), a[j]);
        put(row + m.b(j), b[j]);
      }
  }
}

// cosines and sines of a token's angles; 1 and 0 for pairs that do not turn
template <int NT, bool NEAR, int FORM>
__device__ __forceinline__ void angles(const QkNormParams& p, int64_t b, int64_t t, const Pairs<NT, NEAR, FORM>& m, float (&c)[8], float (&s)[8]) {
  double pos = 0.0;
  if (p.R > 0) {
    const int64_t at = b * p.pos_b + t * p.pos_t;
    pos = p.wide ? (double)global_in<int64_t>(p.positions)[at] : (double)global_in<int32_t>(p.positions)[at];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = m.frequency(j);
    c[j] = 1.f;
    s[j] = 0.f;
    if (i < p.R / 2) {
      const double turns = pos * (double)global_in<float>(p.inv_freq)[i] * 0.15915494309189533577;   // 1 / (2 pi)
      sincospif((float)(2.0 * (turns - rint(turns))), &s[j], &c[j]);
    }
  }
}

template <int NT> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = 1; d < NT; d <<= 1) x += __shfl_xor(x, d);
  return x;
}

template <int NT, bool NEAR, int FORM>
__device__ __forceinline__ void load_weight(const void* w, int wdtype, const Pairs<NT, NEAR, FORM>& m, float (&a)[8], float (&b)[8]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = b[j] = 1.f;
  } else if (wdtype == KDA_DTYPE_BF16) load_pairs<uint16_t>(global_in<uint16_t>(w), m, a, b);
  else load_pairs<float>(global_in<float>(w), m, a, b);
}

template <typename T> __device__ __forceinline__ GlobalPtr<T> row_of(const void* p, kda_stride_t s, int64_t b, int h, int64_t t) {
  return (GlobalPtr<T>)p + b * s.b + h * s.h + t * s.t;
}

// One workgroup: 256 / NT tokens and up to `heads` heads of one tensor.  Blocks of the queries come first.
template <typename T, int NT, bool NEAR, int FORM>
__global__ __launch_bounds__(256) void qk_norm_fwd_kernel(QkNormParams p, int heads, int parts_q, int parts) {
  constexpr int TOK = 256 / NT;
  const int part = blockIdx.x % parts, which = part >= parts_q;
  const int h0 = (which ? part - parts_q : part) * heads, h1 = h0 + heads < p.H[which] ? h0 + heads : p.H[which];
  const uint32_t row = (blockIdx.x / parts) * TOK + threadIdx.x / NT, T_ = (uint32_t)p.T;
  if (row >= (uint32_t)(p.B * p.T)) return;
  const int64_t b = row / T_, t = row - b * T_;
  const Pairs<NT, NEAR, FORM> m((int)(threadIdx.x % NT), p.D, p.R);
  float wa[8], wb[8], c[8], s[8];
  load_weight(p.weight[which], p.wdtype, m, wa, wb);
  angles(p, b, t, m, c, s);
  for (int h = h0; h < h1; ++h) {
    float x[8], y[8];
    load_pairs<T>(row_of<const T>(p.x[which], p.sx[which], b, h, t), m, x, y);
    float r = p.scale[which];
    if (p.norm) {
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) q += m.counts(j) ? x[j] * x[j] + y[j] * y[j] : 0.f;
      r *= rsqrtf(row_sum<NT>(q) / (float)p.D + p.eps);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = x[j] * wa[j] * r, v = y[j] * wb[j] * r;
      x[j] = u * c[j] - v * s[j];
      y[j] = v * c[j] + u * s[j];
    }
    store_pairs<T>(row_of<T>(p.y[which], p.sy[which], b, h, t), m, x, y);
  }
}

// blocks_q workgroups walk the queries' (tokens, heads) items, the others the keys'.  Registers for four wavefronts a SIMD:
// with two more a lane there were three, and 16384 + 16384 rows' heads took 59 us in place of 49.  For it the 16-byte forms keep
// two to five registers in scratch.
template <typename T, int NT, bool NEAR, int FORM>
__global__ __launch_bounds__(256, FORM != kSingle ? 4 : 1) void qk_norm_bwd_kernel(QkNormParams p, int heads, int blocks_q) {
  constexpr int TOK = 256 / NT;
  __shared__ float acc[4][NT * 16];
  const int which = (int)blockIdx.x >= blocks_q;
  const int block = which ? blockIdx.x - blocks_q : blockIdx.x, blocks = which ? gridDim.x - blocks_q : blocks_q;
  const Pairs<NT, NEAR, FORM> m((int)(threadIdx.x % NT), p.D, p.R);
  const uint32_t rows = (uint32_t)(p.B * p.T), T_ = (uint32_t)p.T;
  const int parts = (p.H[which] + heads - 1) / heads;
  const int64_t items = (int64_t)((rows + TOK - 1) / TOK) * parts;
  float wa[8], wb[8], da[8], db[8];
  load_weight(p.weight[which], p.wdtype, m, wa, wb);
#pragma unroll
  for (int j = 0; j < 8; ++j) da[j] = db[j] = 0.f;
  for (int64_t item = block; item < items; item += blocks) {
    const int h0 = (int)(item % parts) * heads, h1 = h0 + heads < p.H[which] ? h0 + heads : p.H[which];
    const uint32_t row = (uint32_t)(item / parts) * TOK + threadIdx.x / NT;
    if (row >= rows) continue;
    const int64_t b = row / T_, t = row - b * T_;
    float c[8], s[8];
    angles(p, b, t, m, c, s);
    for (int h = h0; h < h1; ++h) {
      float x[8], y[8], u[8], v[8];
      load_pairs<T>(row_of<const T>(p.x[which], p.sx[which], b, h, t), m, x, y);
      load_pairs<T>(row_of<const T>(p.dy[which], p.sdy[which], b, h, t), m, u, v);
      float r = 1.f;
      if (p.norm) {
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) q += m.counts(j) ? x[j] * x[j] + y[j] * y[j] : 0.f;
        r = rsqrtf(row_sum<NT>(q) / (float)p.D + p.eps);
      }
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = u[j] * p.scale[which], f = v[j] * p.scale[which];
        u[j] = e * c[j] + f * s[j];
        v[j] = f * c[j] - e * s[j];
        x[j] *= r;
        y[j] *= r;
        da[j] += u[j] * x[j];
        db[j] += v[j] * y[j];
        u[j] *= wa[j];
        v[j] *= wb[j];
        dot += m.counts(j) ? u[j] * x[j] + v[j] * y[j] : 0.f;
      }
      if (p.norm) {
        dot = row_sum<NT>(dot) / (float)p.D;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u[j] = r * (u[j] - x[j] * dot);
          v[j] = r * (v[j] - y[j] * dot);
        }
      }
      store_pairs<T>(row_of<T>(p.dx[which], p.sdx[which], b, h, t), m, u, v);
    }
  }
  if (!p.dweight[which]) return;
  // the wavefront's tokens, then the wavefronts
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int d = NT; d < 64; d <<= 1) {
      da[j] += __shfl_xor(da[j], d);
      db[j] += __shfl_xor(db[j], d);
    }
  }
  if ((threadIdx.x & 63) < NT) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[threadIdx.x >> 6][m.t * 16 + j] = da[j];
      acc[threadIdx.x >> 6][m.t * 16 + 8 + j] = db[j];
    }
  }
  __syncthreads();
  if (threadIdx.x < NT) {
    const auto out = as_global(p.partial) + ((int64_t)which * kMaxBlocks + block) * p.D;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!m.counts(j)) continue;
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        a += acc[w][m.t * 16 + j];
        b += acc[w][m.t * 16 + 8 + j];
      }
      out[m.a(j)] = a;
      out[m.b(j)] = b;
    }
  }
}

// adds up the workgroups' sums: 16 columns a workgroup, 64 threads along the workgroups of each
__global__ __launch_bounds__(1024) void qk_norm_weight_kernel(QkNormParams p, int blocks_q, int blocks_k) {
  __shared__ float part[64][17];
  const int c = threadIdx.x & 15, y = threadIdx.x >> 4, col = blockIdx.x * 16 + c, which = blockIdx.y;
  if (!p.dweight[which]) return;
  const int blocks = which ? blocks_k : blocks_q;
  const auto in = global_in<float>(p.partial) + (int64_t)which * kMaxBlocks * p.D;
  float s = 0.f;
  if (col < p.D) {
#pragma unroll 8
    for (int i = y; i < blocks; i += 64) s += in[(int64_t)i * p.D + col];
  }
  part[y][c] = s;
  __syncthreads();
  if (y == 0 && col < p.D) {
    s = 0.f;
    for (int i = 0; i < 64; ++i) s += part[i][c];
    if (p.wdtype == KDA_DTYPE_BF16) put(global_out<uint16_t>(p.dweight[which]) + col, s);
    else put(global_out<float>(p.dweight[which]) + col, s);
  }
}

template <typename T, int NT, bool NEAR, int FORM>
hipError_t launch_one(const QkNormParams& p, hipStream_t s, bool bwd) {
  constexpr int TOK = 256 / NT;
  const int64_t groups = (p.B * p.T + TOK - 1) / TOK;
  // heads a workgroup walks with one set of angles: as many as leave 8 workgroups a compute unit
  const int64_t all = groups * (p.H[0] + p.H[1]), most = p.H[0] > p.H[1] ? p.H[0] : p.H[1];
  const int heads = (int)(all / 2048 < 1 ? 1 : all / 2048 < most ? all / 2048 : most);
  const int64_t parts_q = (p.H[0] + heads - 1) / heads, parts_k = (p.H[1] + heads - 1) / heads;
  if (!bwd) {
    const int64_t grid = groups * (parts_q + parts_k);
    if (grid > 0)
      hipLaunchKernelGGL((qk_norm_fwd_kernel<T, NT, NEAR, FORM>), dim3((unsigned)grid), dim3(256), 0, s, p, heads, (int)parts_q, (int)(parts_q + parts_k));
    return hipGetLastError();
  }
  const auto blocks = [&](int64_t items) { return (int)(items < kMaxBlocks ? items : kMaxBlocks); };
  const int blocks_q = blocks(groups * parts_q), blocks_k = blocks(groups * parts_k);
  if (blocks_q + blocks_k > 0)
    hipLaunchKernelGGL((qk_norm_bwd_kernel<T, NT, NEAR, FORM>), dim3(blocks_q + blocks_k), dim3(256), 0, s, p, heads, blocks_q);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.dweight[0] && !p.dweight[1])) return e;
  hipLaunchKernelGGL(qk_norm_weight_kernel, dim3((unsigned)((p.D + 15) / 16), 2), dim3(1024), 0, s, p, blocks_q, blocks_k);
  return hipGetLastError();
}

// lanes along a row
template <typename T, bool NEAR, int FORM>
hipError_t launch_d(const QkNormParams& p, hipStream_t s, bool bwd) {
  const int turning = NEAR ? p.D / 2 : p.R / 2, lanes = (turning + 7) / 8 + (p.D / 2 - turning + 7) / 8;
  if (lanes <= 4) return launch_one<T, 4, NEAR, FORM>(p, s, bwd);
  if (lanes <= 8) return launch_one<T, 8, NEAR, FORM>(p, s, bwd);
  if (lanes <= 16) return launch_one<T, 16, NEAR, FORM>(p, s, bwd);
  if (lanes <= 32) return launch_one<T, 32, NEAR, FORM>(p, s, bwd);
  return launch_one<T, 64, NEAR, FORM>(p, s, bwd);
}

template <typename T, bool NEAR> hipError_t launch_form(const QkNormParams& p, hipStream_t s, bool bwd) {
  const int turning = NEAR ? p.D / 2 : p.R / 2, rest = p.D / 2 - turning;
  if (turning % 8 == 0 && rest % 8 == 0) return launch_d<T, NEAR, kWhole>(p, s, bwd);
  // 65 groups do not fit a wavefront
  const bool over = (turning == 0 || turning >= 8) && (rest == 0 || rest >= 8) && (turning + 7) / 8 + (rest + 7) / 8 <= 64;
  return over ? launch_d<T, NEAR, kOver>(p, s, bwd) : launch_d<T, NEAR, kSingle>(p, s, bwd);
}

template <typename T> hipError_t launch_t(const QkNormParams& p, hipStream_t s, bool bwd) {
  return p.interleaved ? launch_form<T, true>(p, s, bwd) : launch_form<T, false>(p, s, bwd);
}

}  // namespace

size_t qk_norm_bwd_workspace_bytes(const QkNormParams& p) { return (size_t)2 * kMaxBlocks * p.D * 4; }
hipError_t launch_qk_norm_fwd(const QkNormParams& p, hipStream_t s) {
  return p.dtype == KDA_DTYPE_BF16 ? launch_t<uint16_t>(p, s, false) : launch_t<float>(p, s, false);
}
hipError_t launch_qk_norm_bwd(const QkNormParams& p, hipStream_t s) {
  return p.dtype == KDA_DTYPE_BF16 ? launch_t<uint16_t>(p, s, true) : launch_t<float>(p, s, true);
}

}  // namespace kda
