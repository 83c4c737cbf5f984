// The walk of linear attention with a decay for each head over one segment (lad_internal.h has the mathematics).
//
// A workgroup owns one (segment, value head) and holds its whole state in registers, in fp32: DZ / 32 wavefronts
// of 32 Z columns each.  Per chunk of 64 tokens, X, Y and Z rows go through LDS once; row tile i of X Y^T
// is formed by wavefront i mod (DZ / 32), decayed, and shared through LDS as planes; then each wavefront forms its
// 32 columns of the outputs and of the new state.
//
// Layouts (lane = 16 g + li).  Products give D tiles: rows 4g .. 4g + 3, column li.  They are formed transposed
// (keys or Z columns along the rows, tokens along the columns), so that
//  - the state's tiles (rows: X channels, columns: Z columns) are operands of the outputs as they lie in registers,
//    with the contraction places of a step of 32 channels in the order {4g + r, 16 + 4g + r};
//  - the tiles of Y X^T (rows: keys) are operands of the products with Z, lane by lane;
//  - a lane has 8 consecutive Z columns of one token: tile c (0, 1) of a wavefront has column 8 (m / 4) + 4 c + m % 4
//    at place m, one 16-byte access of bf16.
// Key tile j has token 16 j + sigma(m) at place m, sigma(m) = 2 m (m < 8), 2 (m - 8) + 1 (m >= 8): with rows 4 banks
// apart modulo 64, the 8 rows that half a wavefront's transposing read touches then lie on different banks.
//
// What bounds it, at 128 x 128 in bf16: chunks of one segment follow one another, 5 us each where a workgroup is alone (130
// tokens of 4 heads: 21 us), 8.6 us with two workgroups on a compute unit.  64K tokens of 16 heads: outputs 276 us (4.1 TB/s, matrix
// cores 30 % busy, the rest vector work on planes and trips to LDS), states 132 us, 4.1 a chunk; the gradients' three walks of
// 2 x 4096 tokens 127 us (in a trace, each kernel on an idle machine).  Two workgroups a compute unit take each other's barriers
// and trips to memory behind their products (with rows read without branches: 64K tokens' forward 540 -> 490 us).
#pragma once

#include "lad_internal.h"

namespace kda {

namespace lad {

typedef short short8 __attribute__((ext_vector_type(8)));
constexpr int kC = kGdrChunk;
enum { kStates, kOuts, kDots, kParts };

__device__ __forceinline__ int sigma(int m) { return m < 8 ? 2 * m : 2 * (m - 8) + 1; }
__device__ __forceinline__ int zcol(int c, int m) { return 8 * (m >> 2) + 4 * c + (m & 3); }

__device__ __forceinline__ floatx4 mac(bf16x8 a, bf16x8 b, floatx4 c) { return mfma(a, b, c); }
__device__ __forceinline__ floatx4 mac(const float8v& a, const float8v& b, floatx4 c) { return mma(a, b, c); }

// A value that the compiler may not carry over from before: addresses made from it are formed where they are used and do not
// keep registers through the loop.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}
// The compiler's schedule puts an LDS read right in front of its use, whose latency a wavefront then waits for (45 times a
// chunk): reads are asked for a step ahead, and nothing crosses this.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// Vector work on x stays behind this, and what made x before it: in its place between the matrix instructions.
__device__ __forceinline__ void from_here(float& x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ void from_here(bf16x8& x, int i) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 w = __builtin_bit_cast(u32x4, x);
  uint32_t v = w[i];
  asm volatile("" : "+v"(v));
  w[i] = v;
  x = __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ void from_here(float8v& x, int i) {
  float a = x[2 * i], b = x[2 * i + 1];
  asm volatile("" : "+v"(a), "+v"(b));
  x[2 * i] = a;
  x[2 * i + 1] = b;
}
template <int N> __device__ __forceinline__ void until_here(Planes<N>& x, int i) {
#pragma unroll
  for (int n = 0; n < N; ++n) from_here(x.p[n], i);
}
__device__ __forceinline__ void until_here(float8v& x, int i) { from_here(x, i); }
// N matrix instructions with V vector ones behind each, which run while it does.
template <int N, int V> __device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
  }
}

// c[i] += a[i] b over planes of one side; the accumulators in turn, so that no product waits for the one before
template <int N> __device__ __forceinline__ void mac2(const Planes<N> (&a)[2], bf16x8 b, floatx4 (&c)[2]) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n)
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = mfma(a[i].p[n], b, c[i]);
}
template <int N> __device__ __forceinline__ void mac2(const bf16x8 (&a)[2], const Planes<N>& b, floatx4 (&c)[2]) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n)
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = mfma(a[i], b.p[n], c[i]);
}
template <int N> __device__ __forceinline__ void mac2(bf16x8 a, const Planes<N> (&b)[2], floatx4 (&c)[2]) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n)
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = mfma(a, b[i].p[n], c[i]);
}
__device__ __forceinline__ void mac2(const float8v (&a)[2], const float8v& b, floatx4 (&c)[2]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i][e], b[e], c[i], 0, 0, 0);
}
__device__ __forceinline__ void mac2(const float8v& a, const float8v (&b)[2], floatx4 (&c)[2]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[i][e], c[i], 0, 0, 0);
}

// Values as planes of bf16, two at a time: a wider conversion compiles to one instruction a value.  Pair i of 8 values.
template <int N> __device__ __forceinline__ void planes_pair(Planes<N>& out, int i, float a, float b) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int n = 0; n < N; ++n) {
    u32x4 p = __builtin_bit_cast(u32x4, out.p[n]);
    const uint32_t h = pk_bf16(a, b);
    p[i] = h;
    out.p[n] = __builtin_bit_cast(bf16x8, p);
    if (n + 1 < N) {
      a -= lo_bf16(h);
      b -= hi_bf16(h);
    }
  }
}
template <int> __device__ __forceinline__ void planes_pair(float8v& out, int i, float a, float b) {
  out[2 * i] = a;
  out[2 * i + 1] = b;
}
template <int N> __device__ __forceinline__ Planes<N> planes_of(const float8v& x, uint16_t) {
  Planes<N> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) planes_pair<N>(r, i, x[2 * i], x[2 * i + 1]);
  return r;
}
template <int N> __device__ __forceinline__ float8v planes_of(const float8v& x, float) { return x; }
// pair i of 8 values of a row
__device__ __forceinline__ float2v widen2(bf16x8 f, int i) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const uint32_t w = __builtin_bit_cast(u32x4, f)[i];
  return float2v{lo_bf16(w), hi_bf16(w)};
}
__device__ __forceinline__ float2v widen2(const float8v& f, int i) { return float2v{f[2 * i], f[2 * i + 1]}; }
__device__ __forceinline__ bf16x8 round8(floatx4 a, floatx4 b) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(bf16x8, u32x4{pk_bf16(a[0], a[1]), pk_bf16(a[2], a[3]), pk_bf16(b[0], b[1]), pk_bf16(b[2], b[3])});
}
__device__ __forceinline__ float8v widen(bf16x8 f, uint16_t) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 w = __builtin_bit_cast(u32x4, f);
  return float8v{lo_bf16(w[0]), hi_bf16(w[0]), lo_bf16(w[1]), hi_bf16(w[1]), lo_bf16(w[2]), hi_bf16(w[2]), lo_bf16(w[3]), hi_bf16(w[3])};
}
__device__ __forceinline__ float8v widen(const float8v& f, float) { return f; }

// A chunk's rows in LDS.
template <typename T, int D> struct Tile {
  static constexpr int kLd = sizeof(T) == 2 ? D + 8 : D + 4;
  using In = typename Frags<T>::In;
  T x[kC * kLd];
  __device__ __forceinline__ void put8(int row, int c, const In& v) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<In*>(x + row * kLd + c) = v;
    else {
      *reinterpret_cast<floatx4*>(x + row * kLd + c) = floatx4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<floatx4*>(x + row * kLd + c + 4) = floatx4{v[4], v[5], v[6], v[7]};
    }
  }
  // The same for rows that are read by row_pair only: bf16 values {4g + r, 16 + 4g + r} of 32 lie side by side, one read in
  // place of two with addresses of their own.
  __device__ __forceinline__ void put8_paired(int row, int c, const In& v) {
    if constexpr (sizeof(T) == 2) {
      T* at = x + row * kLd + (c & ~31) + (c & 8) * 2 + (c & 16) / 4;
      const bf16x4 lo = __builtin_shufflevector(__builtin_bit_cast(short8, v), __builtin_bit_cast(short8, v), 0, 1, 2, 3);
      const bf16x4 hi = __builtin_shufflevector(__builtin_bit_cast(short8, v), __builtin_bit_cast(short8, v), 4, 5, 6, 7);
      *reinterpret_cast<bf16x4*>(at) = lo;
      *reinterpret_cast<bf16x4*>(at + 8) = hi;
    } else put8(row, c, v);
  }
  __device__ __forceinline__ In row_pair(int row, int ks, int g) const {
    if constexpr (sizeof(T) == 2) return *reinterpret_cast<const In*>(x + row * kLd + 32 * ks + 8 * g);
    else return row_frag(row, ks, g);
  }
  // row `row`, channels {32 ks + 4g + r, 32 ks + 16 + 4g + r}
  __device__ __forceinline__ In row_frag(int row, int ks, int g) const {
    const T* at = x + row * kLd + 32 * ks + 4 * g;
    if constexpr (sizeof(T) == 2) {
      const bf16x4 lo = ld4(at), hi = ld4(at + 16);
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const floatx4 a = *reinterpret_cast<const floatx4*>(at), b = *reinterpret_cast<const floatx4*>(at + 16);
      return float8v{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }
  // lane li has, at column col0 + 4 step (li / 4) + li % 4, the tokens of places 4g .. 4g + 3 of key tiles 2 ks, 2 ks + 1
  template <int STEP> __device__ __forceinline__ In columns(int col0, int ks, int lane) const {
    const int li = lane & 15, g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
      typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
      const T* at = x + (32 * ks + sigma(4 * g + (li >> 2))) * kLd + col0 + 4 * STEP * (li & 3);
      const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_bf16x4*)at);
      const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_bf16x4*)(at + 16 * kLd));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      float8v f;
      const T* at = x + (32 * ks + sigma(4 * g)) * kLd + col0 + 4 * STEP * (li >> 2) + (li & 3);   // sigma(4g + r) = sigma(4g) + 2r
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f[r] = at[2 * r * kLd];
        f[4 + r] = at[(16 + 2 * r) * kLd];
      }
      return f;
    }
  }
};

// place of a chunk's token in the order of key tiles
__device__ __forceinline__ int key_place(int t) { return (t & 48) + ((t & 15) >> 1) + ((t & 1) << 3); }

// by key_place of the chunk's tokens
struct Gates {
  float hi[kC], lo[kC];     // the prefix as a sum of two floats: differences stay exact beside a reset
  float oc[kC], uc[kC];     // e^{P} out_scale,  e^{Ptot - P} in_scale
  float tot;                // e^{Ptot}
  double tot2;              // Ptot, in units of ln 2
};

template <typename T, int DX, int DZ, int PL, int MODE> struct Lds {
  static constexpr int kWaves = DZ / 32;
  // A wavefront's part of out . dot, 32 columns: in fp32 where the decay's gradient is rounded to bf16, whose step is far above
  // what these sums lose; added up over the wavefronts and the tokens in double.
  using Dot = std::conditional_t<sizeof(T) == 4 || PL == 3, double, float>;
  Tile<T, DX> y;
  Tile<T, DZ> z;
  Gates gates[2][kWaves];
  struct Outs {
    Tile<T, DX> x;
    char p[4][2][op_frag<T, PL>()];
  };
  struct None {};
  std::conditional_t<MODE != kStates, Outs, None> o;
  Dot dots[MODE >= kDots ? 2 : 0][kWaves][kC];
};

// Memory is read and written through buffer descriptors over a chunk's rows: an offset behind them reads zeros and writes
// nothing, so that rows behind a sequence's end need no branch, and the waits for loads under way count exactly
// what lies behind them.  A chunk's rows lie within 2^31 bytes.
typedef __amdgpu_buffer_rsrc_t Buffer;
typedef unsigned int u32x4v __attribute__((ext_vector_type(4)));
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ Buffer buffer(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, 0x7fffffff, 0x00020000);
}
// 8 values at `at` (of a lane) + `more` (of the wavefront)
__device__ __forceinline__ bf16x8 buffer_row8(Buffer b, uint32_t at, uint32_t more, uint16_t) {
  return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, (int)more, 0));
}
__device__ __forceinline__ float8v buffer_row8(Buffer b, uint32_t at, uint32_t more, float) {
  const floatx4 lo = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, (int)more, 0));
  const floatx4 hi = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, (int)more + 16, 0));
  return float8v{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}
__device__ __forceinline__ uint16_t buffer_one(Buffer b, uint32_t at, uint16_t) { return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, (int)at, 0, 0); }
__device__ __forceinline__ float buffer_one(Buffer b, uint32_t at, float) { return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, (int)at, 0, 0)); }
template <typename V> __device__ __forceinline__ void buffer_put16(Buffer b, uint32_t at, V x, int more = 0) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, x), b, (int)at, more, 0);
}

// one chunk's rows under way from memory
template <typename T, int D, int THREADS> struct Rows8 {
  static constexpr int kPieces = D / 8, kLoads = kC * kPieces / THREADS, kStep = THREADS / kPieces;
  static_assert(THREADS % kPieces == 0 && kLoads * kStep == kC, "whole rows");
  using In = typename Frags<T>::In;
  In v[kLoads];
  // Part `part` of four of a chunk's loads.  Chunk row `row` is memory row `row`, or have - 1 - row backwards; rows
  // `have` and more are zeros.
  __device__ __forceinline__ void load(int part, Buffer b, uint32_t stride, int have, int reverse, int tid) {
    const int id = fresh(tid), r = id / kPieces, rs = reverse ? -1 : 1;
    const uint32_t at = (uint32_t)((reverse ? have - 1 : 0) + rs * r) * stride + id % kPieces * 8 * (int)sizeof(T);
#pragma unroll
    for (int i = part * kLoads / 4; i < (part + 1) * kLoads / 4; ++i)
      v[i] = buffer_row8(b, r < have - i * kStep ? at + (uint32_t)(rs * i * kStep) * stride : kNowhere, 0u, T{});
  }
  template <bool PAIRED = false> __device__ __forceinline__ void leave(Tile<T, D>& t, int id) {
    const int tid = fresh(id);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if constexpr (PAIRED) t.put8_paired(i * kStep + tid / kPieces, tid % kPieces * 8, v[i]);
      else t.put8(i * kStep + tid / kPieces, tid % kPieces * 8, v[i]);
    }
  }
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// 2^(hi + lo), lo a rounding's size beside hi: an exponent of -20 as one float would be off by 6e-7 of the power
__device__ __forceinline__ float exp2_two(float hi, float lo) { return exp2_fast(hi) * (1.f + lo * kLn2); }
__device__ __forceinline__ float exp2_of(double x) {
  const float hi = (float)x;
  return exp2_two(hi, (float)(x - (double)hi));
}

// One wavefront: the gates of a chunk from its lanes' log-decays (0 behind the end), prefixes in units of ln 2.
__device__ __forceinline__ void put_gates(Gates& out, float g, int lane, int reverse, float out_scale, float in_scale) {
  const double own = (double)g * 1.4426950408889634074;
  double p = lane_prefix(own);
  const double tot = last_lane(p);
  p -= reverse ? own : 0.0;
  const float hi = (float)p, lo = (float)(p - (double)hi);
  const int place = key_place(lane);
  out.hi[place] = hi;
  out.lo[place] = lo;
  out.oc[place] = exp2_two(hi, lo) * out_scale;
  out.uc[place] = exp2_of(tot - p) * in_scale;
  out.tot = exp2_of(tot);
  out.tot2 = tot;
}

}  // namespace lad

// PL: planes of the state and of X Y^T in the outputs; UP: of Z in the new state.  Two (off by 2^-17) where only results
// in bf16 are taken from them, three (fp32's accuracy) for states and decays' gradients in fp32.
// MODE: what a walk leaves behind.  kStates: the segment's state from zero and nothing else; kOuts: outputs of type T;
// kDots: also their products with rows of another tensor; kParts: the same with outputs that may be in fp32.
template <typename T, int DX, int DZ, int UP, int PL, int MODE>
__device__ __forceinline__ void lad_walk(const LadParams& p, char* raw, uint32_t unit, uint32_t part) {
  using namespace lad;
  constexpr bool OUT = MODE != kStates, DOTS = MODE >= kDots;
  constexpr int THREADS = 2 * DZ, NW = DZ / 32, MT = DX / 16, KS = DX / 32;
  using In = typename Frags<T>::In;
  auto& lds = *reinterpret_cast<Lds<T, DX, DZ, PL, MODE>*>(raw);
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63, li = lane & 15, g = lane >> 4;

  const uint32_t n_kh = (uint32_t)(p.Hv / p.grp);
  const LadWalk& wk = p.walk[part / (uint32_t)p.grp];
  const int64_t slot = unit / n_kh;
  const int h = (int)(unit % n_kh * (uint32_t)p.grp + part % (uint32_t)p.grp);
  LadSeg sg;
  if (!lad_find(p.seq_start, p.T, p.L, p.n_seq, slot, &sg)) return;
  const int reverse = wk.reverse;
  const int64_t first = sg.seg * p.L;                                    // of the sequence
  const int64_t len = sg.len - first < p.L ? sg.len - first : p.L;       // this segment's tokens
  const bool end = reverse ? sg.seg == 0 : sg.seg == sg.n_seg - 1;       // no segment behind it in the walk's order
  if (wk.skip_end && end) return;

  // chunk c of the walk: its first token in memory, and its tokens.  Backwards the chunks are the same ones.
  // Without outputs the chunks are taken from the end: the state is a sum in which each has the decay behind it.
  const int64_t n_chunks = (len + kC - 1) / kC;
  const bool down = (reverse != 0) == OUT;
  const auto chunk_at = [&](int64_t c) { return sg.t0 + first + kC * (down ? n_chunks - 1 - c : c); };
  const auto chunk_have = [&](int64_t c) {
    const int64_t left = len - kC * (down ? n_chunks - 1 - c : c);
    return (int)(left < kC ? left : kC);
  };
  // the first token of the sequence's part of a tensor; a chunk's rows from there
  const auto rows_of = [&](const void* t, kda_stride_t s, int grp) { return static_cast<const T*>(t) + sg.row * s.b + (h / grp) * s.h; };
  const T* xb = OUT ? rows_of(wk.x, wk.sx, wk.grp_x) : nullptr;
  const T *yb = rows_of(wk.y, wk.sy, wk.grp_y), *zb = rows_of(wk.z, wk.sz, wk.grp_z);
  const int64_t xs = wk.sx.t, ys = wk.sy.t, zs = wk.sz.t;
  constexpr uint32_t E = sizeof(T);

  Rows8<T, DX, THREADS> rx, ry;
  Rows8<T, DZ, THREADS> rz;
  // Part `part` of four of a tensor's rows of chunk c.  Asked for all at once they would fill the queue of the address
  // unit, and their wavefronts would wait there (a quarter of a chunk's time).
  const auto fetch_x = [&](int64_t c, int part) { rx.load(part, buffer(xb + chunk_at(c) * xs), (uint32_t)xs * E, chunk_have(c), reverse, tid); };
  const auto fetch_y = [&](int64_t c, int part) { ry.load(part, buffer(yb + chunk_at(c) * ys), (uint32_t)ys * E, chunk_have(c), reverse, tid); };
  const auto fetch_z = [&](int64_t c, int part) { rz.load(part, buffer(zb + chunk_at(c) * zs), (uint32_t)zs * E, chunk_have(c), reverse, tid); };
  // Each wavefront forms the gates of one chunk in NW, all at the same time; their values of w are asked for as many
  // chunks before.
  const float head_w = p.w_per_head && p.w ? global_in<float>(p.w)[h] : 0.f;
  const T* wb = static_cast<const T*>(p.w) + (p.w_per_head ? 0 : sg.row * p.sw.b + h * p.sw.h);
  const auto gate_ask = [&](int64_t c) {
    const int have = c < n_chunks ? chunk_have(c) : 0;
    const int64_t t = c < n_chunks ? chunk_at(c) : 0;
    const uint32_t at = (uint32_t)((reverse ? have - 1 : 0) + (reverse ? -1 : 1) * lane) * ((uint32_t)p.sw.t * E);
    return buffer_one(buffer(wb + (p.w_per_head ? 0 : t * p.sw.t)), p.w_per_head || lane >= have ? kNowhere : at, T{});
  };
  const auto gate_of = [&](int64_t c, T asked) {
    float x;
    if constexpr (sizeof(T) == 2) x = bf16_to_f32(asked);
    else x = asked;
    const float g = gdr_gate(p.w_per_head ? head_w : x, p.gate, p.g_min);
    return c < n_chunks && lane < chunk_have(c) ? g : 0.f;
  };

  double behind = 0.0;   // without outputs: the decay behind the chunk, in units of ln 2
  T asked{};
  if (n_chunks > 0) {
    asked = gate_ask(wave);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (OUT) fetch_x(0, i);
      fetch_y(0, i);
      fetch_z(0, i);
    }
  }

  floatx4 S[MT][2];
  {
    const int64_t at = wk.by_slot ? slot * p.Hv + h : sg.seq * p.Hv + h;
    const auto src = global_in<float>(wk.entering) + at * (DX * DZ);
#pragma unroll
    for (int m = 0; m < MT; ++m) S[m][0] = S[m][1] = floatx4{};
    if (wk.entering && wk.transposed) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 2; ++c) S[m][c] = ld4f(src + (32 * wave + zcol(c, li)) * DX + 16 * m + 4 * g);
    } else if (wk.entering) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[m][c][r] = src[(16 * m + 4 * g + r) * DZ + 32 * wave + zcol(c, li)];
    }
  }

  // this wavefront's part of out . dot for every token of the chunk
  using Dot = typename Lds<T, DX, DZ, PL, MODE>::Dot;
  In dots[DOTS ? 4 : 1];
  // row of a chunk in memory = r0 + rs row
  const int rs = reverse ? -1 : 1;
  const auto ask_dots = [&](int64_t c) {
    const int have = chunk_have(c), r0 = reverse ? have - 1 : 0, ln = fresh(lane), li = ln & 15, g = ln >> 4;
    const Buffer b = buffer(rows_of(wk.dot, wk.sdot, wk.grp_dot) + chunk_at(c) * wk.sdot.t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * i + li;
      const uint32_t at = (uint32_t)(r0 + rs * row) * ((uint32_t)wk.sdot.t * E) + (32 * wave + 8 * g) * E;
      dots[i] = buffer_row8(b, wk.dot && row < have ? at : kNowhere, 0u, T{});
    }
  };
  const auto row_dots = [&](const floatx4 (&acc)[4][2], Dot* out) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float8v d = widen(dots[i], T{});
      Dot s = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) s += (Dot)acc[i][0][r] * (Dot)d[r] + (Dot)acc[i][1][r] * (Dot)d[4 + r];
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (g == 0) out[16 * i + li] = s;
    }
  };

  if (n_chunks > 0) {
    put_gates(lds.gates[0][wave], gate_of(wave, asked), lane, reverse, wk.out_scale, wk.in_scale);
    asked = gate_ask(NW + wave);
    if constexpr (OUT) rx.template leave<true>(lds.o.x, tid);
    ry.leave(lds.y, tid);
    rz.leave(lds.z, tid);
  }
  block_barrier();

  for (int64_t c = 0; c < n_chunks; ++c) {
    const int have = chunk_have(c);
    const Gates& gt = lds.gates[c / NW & 1][c % NW];
    if (c % NW == NW - 1) {   // the gates of the next NW chunks
      const int64_t mine = c + 1 + wave;
      put_gates(lds.gates[(c + 1) / NW & 1][wave], gate_of(mine, asked), lane, reverse, wk.out_scale, wk.in_scale);
      asked = gate_ask(mine + NW);
    }
    const int64_t next = c + 1 < n_chunks ? c + 1 : c;   // the last chunk asks for its own rows again

    if constexpr (OUT) {
      // this wavefront's row tiles of the decayed X Y^T, transposed: column li is token 16 i + li.  Two key tiles at a
      // time, the later two only where a row comes behind them.
#pragma unroll
      for (int ii = 0; ii < 4 / NW; ++ii) {
        const int i = wave + ii * NW, ln = fresh(lane), li = ln & 15, g = ln >> 4;
        const auto key_tiles = [&](int half) {
          floatx4 t[2] = {};
          In xf[2], yf[2][2];
          const auto ask = [&](int ks) {
            xf[ks & 1] = lds.o.x.row_pair(16 * i + li, ks, g);
#pragma unroll
            for (int j = 0; j < 2; ++j) yf[ks & 1][j] = lds.y.row_frag(32 * half + 16 * j + sigma(li), ks, g);
          };
          ask(0);
          const float qh = gt.hi[16 * i + key_place(li)], ql = gt.lo[16 * i + key_place(li)];
          floatx4 kh[2], kl[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            kh[j] = *reinterpret_cast<const floatx4*>(gt.hi + 32 * half + 16 * j + 4 * g);
            kl[j] = *reinterpret_cast<const floatx4*>(gt.lo + 32 * half + 16 * j + 4 * g);
          }
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            if (ks + 1 < KS) ask(ks + 1);
            in_order();
#pragma unroll
            for (int j = 0; j < 2; ++j) t[j] = mac(yf[ks & 1][j], xf[ks & 1], t[j]);
            in_order();
          }
          // log2 of the decays; those of later keys are put where the exponential is 0: selecting the product would put it behind a branch
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const bool before = 32 * half + 16 * j + sigma(4 * g + r) <= 16 * i + li;
              float e;
              if constexpr (sizeof(T) == 4 || PL == 3) {
                // |qh| >= |kh| there, so what their difference loses is found exactly.  It is of the prefixes' rounding, which
                // behind many resets is far more than that of their difference (32 resets: 0.03), so the two are summed first
                // and what that sum loses is left (without it a reset every second token put outputs off by 2.3e-5).
                const float d = qh - kh[j][r], l = ((qh - d) - kh[j][r]) + (ql - kl[j][r]), sum = d + l;
                e = exp2_two(before ? sum : -1e30f, l - (sum - d));
              } else {
                e = exp2_fast(before ? (qh - kh[j][r]) + (ql - kl[j][r]) : -1e30f);
              }
              t[j][r] *= e * (wk.out_scale * wk.in_scale);
            }
          const float8v f = {t[0][0], t[0][1], t[0][2], t[0][3], t[1][0], t[1][1], t[1][2], t[1][3]};
          store_frag(lds.o.p[i][half], ln, planes_of<PL>(f, T{}));
        };
        key_tiles(0);
        if (i >= 2) key_tiles(1);
      }
    }

    floatx4 acc[4][2];
    if constexpr (OUT) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = floatx4{};
      In xf[2][4];
      typename Frags<T>::template Op<PL> sp[2][2];
      const auto ask = [&](int ks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) xf[ks & 1][i] = lds.o.x.row_pair(16 * i + li, ks, g);
      };
      const float tot = gt.tot;
      // planes of the state, pairs 2 u and 2 u + 1 of its 8 in step ks; it is not needed as it was any more
      const auto planes = [&](int ks, int u) {
#pragma unroll
        for (int k = 2 * u; k < 2 * u + 2; ++k) {
          const int cc = k >> 2, i = k & 3;
          floatx4& from = S[2 * ks + (i >> 1)][cc];
          float a = from[2 * (i & 1)], b = from[2 * (i & 1) + 1];
          from_here(a);
          from_here(b);
          planes_pair<PL>(sp[ks & 1][cc], i, a, b);
          a *= tot;
          b *= tot;
          until_here(sp[ks & 1][cc], i);
          from_here(a);
          from_here(b);
          from[2 * (i & 1)] = a;
          from[2 * (i & 1) + 1] = b;
        }
      };
      ask(0);
#pragma unroll
      for (int u = 0; u < 4; ++u) planes(0, u);
      in_order();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (ks + 1 < KS) ask(ks + 1);
#pragma unroll
        for (int i = ks * 4 / KS; i < (ks + 1) * 4 / KS; ++i) {
          fetch_x(next, i);
          fetch_y(next, i);
        }
        in_order();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mac2(sp[ks & 1], xf[ks & 1][i], acc[i]);
          if (ks + 1 < KS) {
            planes(ks + 1, i);
            interleave<2 * PL, 4>();
          }
          in_order();
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float oc = gt.oc[16 * i + key_place(li)];
        acc[i][0] *= oc;
        acc[i][1] *= oc;
      }
    }

    // the new state, and the rest of the outputs: both take the columns of Z
    In zf[2];
    const auto ask_z = [&](int ks) {
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) zf[cc] = lds.z.template columns<2>(32 * wave + 4 * cc, ks, lane);
    };
    const float before = OUT ? 1.f : exp2_of(behind);
    behind += gt.tot2;
    typename Frags<T>::template Op<UP> zu[2][2];
    float8v u;
    const auto ask_u = [&](int ks) {
      const floatx4 u0 = *reinterpret_cast<const floatx4*>(gt.uc + 32 * ks + 4 * g), u1 = *reinterpret_cast<const floatx4*>(gt.uc + 32 * ks + 16 + 4 * g);
      u = float8v{u0[0], u0[1], u0[2], u0[3], u1[0], u1[1], u1[2], u1[3]};
      if constexpr (!OUT) {
#pragma unroll
        for (int r = 0; r < 8; ++r) u[r] *= before;
      }
    };
    const auto decayed = [&](int ks, int k) {   // pair k of the 8 of Z's columns
      from_here(zf[k >> 2], k & 3);
      const float2v f = widen2(zf[k >> 2], k & 3);
      planes_pair<UP>(zu[ks][k >> 2], k & 3, f[0] * u[2 * (k & 3)], f[1] * u[2 * (k & 3) + 1]);
      until_here(zu[ks][k >> 2], k & 3);
    };
    if constexpr (!OUT) {   // nothing else lies before it: all at once
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fetch_y(next, i);
        fetch_z(next, i);
      }
    }
    // the steps' columns of Y, asked for two products ahead
    In yf[3];
    const auto ask_y = [&](int n) {
      if (n < 2 * MT) yf[n % 3] = lds.y.template columns<1>(16 * (n % MT), n / MT, lane);
    };
    ask_z(0);
    ask_u(0);
    ask_y(0);
    ask_y(1);
#pragma unroll
    for (int k = 0; k < 8; ++k) decayed(0, k);
    ask_z(1);
    ask_u(1);
    in_order();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (DOTS && ks == 1) ask_dots(c);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int n = ks * MT + m;
        ask_y(n + 2);
        in_order();
        mac2(yf[n % 3], zu[ks], S[m]);
        if (ks == 0) {   // the next step's planes beside this one's products
#pragma unroll
          for (int k = m * 8 / MT; k < (m + 1) * 8 / MT; ++k) decayed(1, k);
          interleave<2 * UP, 4>();
        }
        in_order();
        // a quarter of the rows that are still to be asked for, four times over the two steps
        if (n % (MT / 2) == MT / 2 - 1) {
          if constexpr (OUT) fetch_z(next, n / (MT / 2));
        }
      }
    }
    if constexpr (OUT) ask_z(0);
    if constexpr (OUT) {
      if constexpr (DOTS) row_dots(acc, lds.dots[0][wave]);
      block_barrier();   // the tiles of X Y^T are there
      typename Frags<T>::template Op<PL> pf[2];
      const auto ask = [&](int n) {   // tiles (0..3, 0), (2..3, 1)
        const int i = n < 4 ? n : n - 2, ks = n < 4 ? 0 : 1;
        if (n < 6) pf[n & 1] = load_frag<typename Frags<T>::template Op<PL>>(lds.o.p[i][ks], lane);
      };
      ask(0);
#pragma unroll
      for (int n = 0; n < 6; ++n) {
        ask(n + 1);
        in_order();
        mac2(zf, pf[n & 1], acc[n < 4 ? n : n - 2]);
        if (n == 3) ask_z(1);
        in_order();
      }
      if constexpr (DOTS) row_dots(acc, lds.dots[1][wave]);
      const int64_t out_row = sg.row * wk.so.b + h * wk.so.h + chunk_at(c) * wk.so.t;
      const bool wide = MODE == kParts && wk.out_f32;
      const uint32_t esz = wide ? 4 : E, ostep = (uint32_t)wk.so.t * esz;
      const Buffer ob = buffer(static_cast<char*>(wk.out) + out_row * esz);
      const int r0 = reverse ? have - 1 : 0, ln = fresh(lane), li = ln & 15, g = ln >> 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * i + li;
        const uint32_t at = row < have ? (uint32_t)(r0 + rs * row) * ostep + (32 * wave + 8 * g) * esz : kNowhere;
        if constexpr (sizeof(T) == 2) buffer_put16(ob, wide ? kNowhere : at, round8(acc[i][0], acc[i][1]));
        if constexpr (sizeof(T) == 4 || MODE == kParts) {
          buffer_put16(ob, sizeof(T) == 4 || wide ? at : kNowhere, acc[i][0]);
          buffer_put16(ob, sizeof(T) == 4 || wide ? at : kNowhere, acc[i][1], 16);
        }
      }
    }
    // a state that forgets: what lies further from its end has a factor of 0
    if (!OUT && exp2_fast((float)behind) == 0.f) break;
    block_barrier();   // nobody reads this chunk's rows any more
    if constexpr (OUT) rx.template leave<true>(lds.o.x, tid);
    ry.leave(lds.y, tid);
    rz.leave(lds.z, tid);
    if constexpr (DOTS) {
      if (wk.dot && tid < kC && tid < have) {
        const int64_t at = (sg.row * p.Hv + h) * p.T + chunk_at(c) + (reverse ? have - 1 - tid : tid);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          double s = 0.0;
#pragma unroll
          for (int w = 0; w < NW; ++w) s += lds.dots[k][w][tid];
          wk.dots[k][at] = s;
        }
      }
    }
    block_barrier();
  }

  if (!OUT && wk.decay && tid == 0) wk.decay[slot * p.Hv + h] = exp2_of(behind);
  if (wk.leaving && (wk.leave_slot || end)) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < 2; ++c) settle(S[m][c]);
    const int64_t at = wk.leave_slot ? slot * p.Hv + h : sg.seq * p.Hv + h;
    const auto dst = as_global(wk.leaving) + at * (DX * DZ);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int z = 32 * wave + zcol(c, li), x = 16 * m + 4 * g;
        if (wk.transposed) *repoint<floatx4>(dst + z * DX + x) = S[m][c];
        else {
#pragma unroll
          for (int r = 0; r < 4; ++r) dst[(x + r) * DZ + z] = S[m][c][r];
        }
      }
  }
}

// Workgroups of one (segment, query/key head) read the same rows: they get blocks of one XCD (block b runs on XCD b mod
// 8).  False for a block without work.
__device__ __forceinline__ bool lad_block(const LadParams& p, uint32_t* unit, uint32_t* part) {
  const uint32_t parts = (uint32_t)(p.n_walks * p.grp), round = blockIdx.x >> 3;
  *unit = (blockIdx.x & 7) + 8 * (round / parts);
  *part = round % parts;
  return *unit < (uint32_t)p.slots * (uint32_t)(p.Hv / p.grp);
}

template <typename T, int DX, int DZ, int UP, int PL, int MODE, int OCC>
__global__ __launch_bounds__(2 * DZ, OCC) void lad_walk_kernel(LadParams p) {
  extern __shared__ __attribute__((aligned(16))) char raw[];
  uint32_t unit, part;
  if (lad_block(p, &unit, &part)) lad_walk<T, DX, DZ, UP, PL, MODE>(p, raw, unit, part);
}

// The three walks of the gradients where dk and dv differ: the first two have DX = dv, the third DX = dk.  A launch of its own
// for the third would run behind them (dk = 64, dv = 128 in fp32, 5 sequences of up to 447 tokens: 24 + 17 us).
template <typename T, int DX, int DZ, int UP, int PL, int MODE, int OCC>
__global__ __launch_bounds__(2 * (DX > DZ ? DX : DZ), OCC) void lad_walks_kernel(LadParams p) {
  extern __shared__ __attribute__((aligned(16))) char raw[];
  uint32_t unit, part;
  if (!lad_block(p, &unit, &part)) return;
  if (part < 2 * (uint32_t)p.grp) {
    if (threadIdx.x < 2 * DZ) lad_walk<T, DX, DZ, UP, PL, MODE>(p, raw, unit, part);
  } else {
    if (threadIdx.x < 2 * DX) lad_walk<T, DZ, DX, UP, PL, MODE>(p, raw, unit, part);
  }
}

template <typename T, int DX, int DZ, int UP, int PL, int MODE>
hipError_t launch_walk_one(const LadParams& p, hipStream_t s) {
  constexpr int kOne = (int)sizeof(lad::Lds<T, DX, DZ, PL, MODE>), kOther = (int)sizeof(lad::Lds<T, DZ, DX, PL, MODE>);
  constexpr bool kBoth = MODE >= lad::kDots && DX != DZ;
  constexpr int kLdsBytes = kBoth && kOther > kOne ? kOther : kOne, kSide = kBoth && DX > DZ ? DX : DZ;
  // Two workgroups a compute unit where registers and LDS allow it; a single wavefront's 32 columns beside 128 need more than
  // half of a SIMD's registers for the rows under way.  The gradients of 64 x 128 and 128 x 64 keep 4 and 7 registers in scratch for
  // it (2 x 4096 tokens, 16 heads: 158 and 146 us, with one workgroup 203 and 193); those of 32 x 128 in fp32 do at any rate.
  constexpr int OCC = sizeof(T) == 2 && kSide == 128 && PL == 2 && !(kBoth && DX + DZ == 160) ? 2 : 1;
  void (*kernel)(LadParams);
  if constexpr (kBoth) kernel = lad_walks_kernel<T, DX, DZ, UP, PL, MODE, OCC>;
  else kernel = lad_walk_kernel<T, DX, DZ, UP, PL, MODE, OCC>;
  static std::atomic<uint64_t> done;
  const hipError_t set = set_dyn_lds(reinterpret_cast<const void*>(kernel), kLdsBytes, done);
  if (set != hipSuccess) return set;
  const int64_t grid = gdr_blocks(p.slots * (p.Hv / p.grp), p.n_walks * p.grp);
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(2 * kSide), kLdsBytes, s, p);
  return hipGetLastError();
}

template <typename T, int UP, int PL, int MODE>
hipError_t launch_walk_dims(const LadParams& p, int dx, int dz, hipStream_t s) {
  switch (dx * 256 + dz) {
    case 32 * 256 + 32: return launch_walk_one<T, 32, 32, UP, PL, MODE>(p, s);
    case 32 * 256 + 64: return launch_walk_one<T, 32, 64, UP, PL, MODE>(p, s);
    case 32 * 256 + 128: return launch_walk_one<T, 32, 128, UP, PL, MODE>(p, s);
    case 64 * 256 + 32: return launch_walk_one<T, 64, 32, UP, PL, MODE>(p, s);
    case 64 * 256 + 64: return launch_walk_one<T, 64, 64, UP, PL, MODE>(p, s);
    case 64 * 256 + 128: return launch_walk_one<T, 64, 128, UP, PL, MODE>(p, s);
    case 128 * 256 + 32: return launch_walk_one<T, 128, 32, UP, PL, MODE>(p, s);
    case 128 * 256 + 64: return launch_walk_one<T, 128, 64, UP, PL, MODE>(p, s);
    default: return launch_walk_one<T, 128, 128, UP, PL, MODE>(p, s);
  }
}

}  // namespace kda
