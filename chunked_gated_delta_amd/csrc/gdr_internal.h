// Internal declarations of the head-gated delta rule (one log-decay per token and head) and of the
// norms around a block: parameters, launchers and the operand fragments of the matrix-core kernels.
//
// Chunk form (C = 64 tokens; per sequence and value head, S entering the chunk, G the chunk's inclusive
// prefix of the log-decay, D_rj = e^{G_r - G_j}, gam = e^G, eta = e^{G_last - G}):
//   A = strict_lower(K K^T . D)      P = scale lower(Q K^T . D)      T' = (I + A diag(beta))^{-1}
//   E = V - gam K S     F = T' E     U = beta F
//   O = scale gam Q S + P U          S <- e^{G_last} S + K^T (eta U)
// One decay per head keeps it out of the operands: K K^T and Q K^T are products of the inputs as they
// are (bf16 products are exact), and every decay factor is at most 1 and multiplies an fp32 result.
#pragma once

#include "kda_mfma_util.h"

namespace kda {

constexpr int kGdrChunk = 64;

struct GdrParams {
  const void *q, *k, *v, *w, *beta;
  kda_stride_t sq, sk, sv, sw, sb;
  const float* S0;              // nullable
  const int32_t* seq_start;     // packed sequences: n_seq + 1 offsets; null: every batch row is a sequence
  int64_t B, T, n_seq;          // n_seq = B when not packed
  int Hk, Hv, dk, dv;
  int dtype, gate;
  float g_min, scale;
  void* o;
  kda_stride_t so;
  float* S_final;               // nullable
  // backward
  const void* dO;
  kda_stride_t sdo;
  const float* dSf;             // nullable
  void *dq, *dk_, *dv_, *dw, *dbeta;
  kda_stride_t sdq, sdk, sdv, sdw, sdb;
  float* dS0;                   // nullable
  // workspace sections, one block per (chunk slot, head); see gdr_layout
  char *ws_gate, *ws_ti, *ws_tt, *ws_p, *ws_s, *ws_ds, *ws_f, *ws_e, *ws_db;
};

struct GdrStepParams {
  const void *q, *k, *v, *w, *beta;
  kda_stride_t sq, sk, sv, sw, sb, so;
  const int32_t* slots;         // null: row b uses state b
  float* S;
  void* o;
  int64_t B, T, n_slots;
  int Hk, Hv, dk, dv;
  int dtype, gate;
  float g_min, scale;
};

struct NormParams {
  const void *x, *z, *res, *weight, *weight2;
  kda_stride_t sx, sz, sr, ss, sy;
  void *s, *y;
  // backward: cotangents and gradients
  const void *ds, *dy;
  void *dx, *dz, *dres, *dweight, *dweight2;
  kda_stride_t sds, sdy, sdx, sdz, sdr;
  float* partial;               // workspace: per-workgroup sums of the weights' gradients
  int64_t B, H, T, D;
  int dtype, wdtype, act;
  float alpha, eps;
};

int64_t gdr_slots(int64_t B, int64_t T, int64_t n_seq, bool packed);
// sets the workspace sections of p from base (may be null) and returns the bytes needed
size_t gdr_layout(GdrParams& p, void* base, bool bwd);
hipError_t launch_gdr_fwd(const GdrParams& p, hipStream_t s);
hipError_t launch_gdr_bwd(const GdrParams& p, hipStream_t s);
hipError_t launch_gdr_prep(const GdrParams& p, hipStream_t s, bool bwd);
hipError_t launch_gdr_scan(const GdrParams& p, hipStream_t s, bool states);
hipError_t launch_gdr_rscan(const GdrParams& p, hipStream_t s);
hipError_t launch_gdr_grad(const GdrParams& p, hipStream_t s);
hipError_t launch_gdr_step(const GdrStepParams& p, hipStream_t s);
size_t norm_bwd_workspace_bytes(const NormParams& p);
hipError_t launch_norm_fwd(const NormParams& p, hipStream_t s);
hipError_t launch_norm_bwd(const NormParams& p, hipStream_t s);

// ---------------------------------------------------------------- workspace blocks

// per (slot, value head), fp32: gam, eta, beta, and G as a sum of two floats (64 each), then e^{G_last}
constexpr int kGateGam = 0, kGateEta = 64, kGateBeta = 128, kGateHi = 192, kGateLo = 256, kGateLast = 320;
constexpr int kGateFloats = 336;
// a 64 x 64 triangular matrix as A operands: 16 x 32 fragments of the row tiles that hold any of it
constexpr int kTriFrags = 6;
__host__ __device__ constexpr int lower_frag(int tile, int ks) { return tile < 2 ? tile : 2 + 2 * (tile - 2) + ks; }
__host__ __device__ constexpr int upper_frag(int tile, int ks) { return tile < 2 ? 2 * tile + ks : 4 + (tile - 2); }

// ---------------------------------------------------------------- sequences and chunk slots

// A packed batch keeps its chunks at slot floor(start / 64) + sequence, which leaves room for every
// sequence's partly filled chunk without a prefix sum over the lengths.  Offsets are clamped into
// [0, T], so that offsets out of order cannot address anything out of range.
struct GdrSeq {
  int64_t row, t0, len, slot0, n_chunks;   // batch row, first token, tokens, first chunk slot, chunks
};

__device__ __forceinline__ int64_t clamp_off(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

__device__ __forceinline__ GdrSeq gdr_seq(const GdrParams& p, int64_t s) {
  GdrSeq q;
  if (!p.seq_start) {
    q.row = s;
    q.t0 = 0;
    q.len = p.T;
    q.n_chunks = (p.T + kGdrChunk - 1) / kGdrChunk;
    q.slot0 = s * q.n_chunks;
  } else {
    const int64_t a = clamp_off(p.seq_start[s], 0, p.T), e = clamp_off(p.seq_start[s + 1], a, p.T);
    q.row = 0;
    q.t0 = a;
    q.len = e - a;
    q.n_chunks = (q.len + kGdrChunk - 1) / kGdrChunk;
    q.slot0 = a / kGdrChunk + s;
  }
  return q;
}

// the sequence whose chunks hold this slot, the chunk in *chunk; false where the slot holds none
__device__ __forceinline__ bool gdr_find(const GdrParams& p, int64_t slot, GdrSeq* seq, int64_t* chunk) {
  int64_t lo = 0;
  if (!p.seq_start) {
    lo = slot / ((p.T + kGdrChunk - 1) / kGdrChunk);
  } else {
    int64_t hi = p.n_seq - 1;   // the last sequence whose first slot is not behind this one
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) / 2;
      if (clamp_off(p.seq_start[mid], 0, p.T) / kGdrChunk + mid <= slot) lo = mid; else hi = mid - 1;
    }
  }
  *seq = gdr_seq(p, lo);
  *chunk = slot - seq->slot0;
  return *chunk >= 0 && *chunk < seq->n_chunks;
}

// log-decay of one gate value.  Below -1e4 it is held there (e^-1e4 is 0 already), so that a decay
// of -infinity, a reset of the state, leaves differences of prefixes defined; NaN stays.
__device__ __forceinline__ float gdr_gate(float w, int gate, float g_min) {
  float g = w;
  if (gate == KDA_GATE_BOUNDED) g = gate_f32(w, g_min, 0);
  if (gate == KDA_GATE_SOFTPLUS) g = gate_f32(w, 0.f, 1);
  return g < -1e4f ? -1e4f : g;
}
// its derivative by w
__device__ __forceinline__ float gdr_gate_grad(float w, int gate, float g_min) {
  if (gate == KDA_GATE_LOG) return 1.f;
  const float s = 1.f / (1.f + expf(-w));
  return gate == KDA_GATE_BOUNDED ? g_min * s * (1.f / (1.f + expf(w))) : -s;
}

// ---------------------------------------------------------------- memory accesses

// Pointers taken from the parameter block are global memory; said in their type, so that their accesses
// are global instructions wherever the pointer went (a flat one would also count as an LDS access, and
// every barrier's wait for LDS would wait for it).
#define KDA_GLOBAL __attribute__((address_space(1)))
template <typename T> using GlobalPtr = KDA_GLOBAL T*;
template <typename T> __device__ __forceinline__ GlobalPtr<T> as_global(T* p) { return (GlobalPtr<T>)p; }
template <typename T> __device__ __forceinline__ GlobalPtr<const T> global_in(const void* p) { return (GlobalPtr<const T>)p; }
template <typename T> __device__ __forceinline__ GlobalPtr<T> global_out(void* p) { return (GlobalPtr<T>)p; }
template <typename To, typename From> __device__ __forceinline__ const To* repoint(const From* p) { return reinterpret_cast<const To*>(p); }
template <typename To, typename From> __device__ __forceinline__ const KDA_GLOBAL To* repoint(const KDA_GLOBAL From* p) {
  return reinterpret_cast<const KDA_GLOBAL To*>(p);
}
template <typename To, typename From> __device__ __forceinline__ To* repoint(From* p) { return reinterpret_cast<To*>(p); }
template <typename To, typename From> __device__ __forceinline__ KDA_GLOBAL To* repoint(KDA_GLOBAL From* p) {
  return reinterpret_cast<KDA_GLOBAL To*>(p);
}
__device__ __forceinline__ float get(const KDA_GLOBAL uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float get(const KDA_GLOBAL float* p) { return *p; }
__device__ __forceinline__ void put(KDA_GLOBAL uint16_t* p, float x) { *p = (uint16_t)pk_bf16(x, x); }
__device__ __forceinline__ void put(KDA_GLOBAL float* p, float x) { *p = x; }
// element `off` (of lanes) behind `base` (of the wavefront): the address needs no vector arithmetic
template <typename T> __device__ __forceinline__ const KDA_GLOBAL T* lane_at(const KDA_GLOBAL T* base, uint32_t bytes) {
  return (const KDA_GLOBAL T*)((const KDA_GLOBAL char*)base + bytes);
}
template <typename T> __device__ __forceinline__ KDA_GLOBAL T* lane_at(KDA_GLOBAL T* base, uint32_t bytes) {
  return (KDA_GLOBAL T*)((KDA_GLOBAL char*)base + bytes);
}
template <typename P> __device__ __forceinline__ floatx4 ld4f(P p) { return *repoint<floatx4>(p); }

// the wavefront's number in its workgroup, known to be the same in all lanes
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// ---------------------------------------------------------------- operand fragments

// A fragment is 8 values a lane: of the A operand row li, of the B operand column li, at contraction
// places 8g .. 8g + 7 (lane = 16 g + li) of a step of 32.  bf16 inputs are one register group, exact.
// Values that the kernels compute are carried as sums of bf16 planes, each the rounding of what the planes
// before it leave: three planes hold an fp32 value whole, two are off by at most 2^-17 of it.  The state,
// its adjoint and everything between them (E, T', U) take three: with two, S_final was off by 4e-6 where
// fp32 arithmetic is off by 5e-8, with three it keeps fp32's accuracy for 1.5 times the matrix
// instructions.  What enters only results of the inputs' type takes two.
// fp32 inputs use v_mfma_f32_16x16x4_f32 on the same 8 values, one place of each lane group at a time.
template <int N> struct Planes {
  bf16x8 p[N];
};
template <typename T> struct Frags;
template <> struct Frags<uint16_t> {
  using In = bf16x8;
  template <int N> using Op = Planes<N>;
  static constexpr int in_planes = 1;
  static constexpr int planes(int n) { return n; }
};
template <> struct Frags<float> {
  using In = float8v;
  template <int N> using Op = float8v;
  static constexpr int in_planes = 2;
  static constexpr int planes(int) { return 2; }
};
constexpr int kPlane = 64 * 16;   // 16 bytes a lane; an fp32 fragment is two planes (places 0-3 and 4-7)
// planes of the states and of F that the backward keeps for its gradients (one of fp32)
template <typename T> constexpr int kKept = sizeof(T) == 2 ? 2 : 1;
template <typename T> constexpr int in_frag() { return Frags<T>::in_planes * kPlane; }
template <typename T, int N> constexpr int op_frag() { return Frags<T>::planes(N) * kPlane; }

__device__ __forceinline__ floatx4 mma(bf16x8 a, bf16x8 b, floatx4 c) { return mfma(a, b, c); }
template <int N> __device__ __forceinline__ floatx4 mma(const Planes<N>& a, bf16x8 b, floatx4 c) {
#pragma unroll
  for (int i = N - 1; i >= 0; --i) c = mfma(a.p[i], b, c);
  return c;
}
__device__ __forceinline__ floatx4 mma(const float8v& a, const float8v& b, floatx4 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

// To be put between a matrix instruction behind a branch and the vector reads of its result: this compiler
// leaves out the wait between them where a branch target lies between (shown in its assembly; the first
// value read was wrong).
__device__ __forceinline__ void settle(floatx4& x) { asm volatile("s_nop 11" : "+v"(x)); }

// acc + sum over steps of a[i] b[i], as chains of their own added at the end: one dependent matrix
// instruction takes 32 cycles, an independent one 16
template <int K, int N> __device__ __forceinline__ floatx4 mma_steps(const bf16x8 (&a)[K], const Planes<N> (&b)[K], floatx4 acc) {
  floatx4 c[N];
#pragma unroll
  for (int n = 1; n < N; ++n) c[n] = floatx4{};
  c[0] = acc;
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) c[n] = mfma(a[i], b[i].p[n], c[n]);
#pragma unroll
  for (int n = N - 1; n > 0; --n) c[n - 1] += c[n];
  return c[0];
}
template <int K> __device__ __forceinline__ floatx4 mma_steps(const float8v (&a)[K], const float8v (&b)[K], floatx4 acc) {
  floatx4 c[2] = {acc, floatx4{}};
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i][e], b[i][e], c[e & 1], 0, 0, 0);
  return c[0] + c[1];
}
// both sides in two planes: the three products above the last plane's size
template <int K> __device__ __forceinline__ floatx4 mma_steps(const Planes<2> (&a)[K], const Planes<2> (&b)[K], floatx4 acc) {
  floatx4 c[3] = {acc, floatx4{}, floatx4{}};
#pragma unroll
  for (int i = 0; i < K; ++i) {
    c[2] = mfma(a[i].p[1], b[i].p[0], c[2]);
    c[1] = mfma(a[i].p[0], b[i].p[1], c[1]);
    c[0] = mfma(a[i].p[0], b[i].p[0], c[0]);
  }
  return c[0] + (c[1] + c[2]);
}
// both sides in three planes: the six products above the last plane's size
template <int K> __device__ __forceinline__ floatx4 mma_steps(const Planes<3> (&a)[K], const Planes<3> (&b)[K], floatx4 acc) {
  floatx4 c[3] = {acc, floatx4{}, floatx4{}};
#pragma unroll
  for (int i = 0; i < K; ++i) {
    c[2] = mfma(a[i].p[1], b[i].p[1], c[2]);
    c[1] = mfma(a[i].p[1], b[i].p[0], c[1]);
    c[0] = mfma(a[i].p[0], b[i].p[0], c[0]);
    c[2] = mfma(a[i].p[2], b[i].p[0], c[2]);
    c[1] = mfma(a[i].p[0], b[i].p[1], c[1]);
    c[2] = mfma(a[i].p[0], b[i].p[2], c[2]);
  }
  return c[0] + (c[1] + c[2]);
}

__device__ __forceinline__ void zero_frag(bf16x8& f) { f = bf16x8{}; }
__device__ __forceinline__ void zero_frag(float8v& f) { f = float8v{}; }

// 8 consecutive values of a row in memory (16-byte aligned)
__device__ __forceinline__ bf16x8 load_row8(const KDA_GLOBAL uint16_t* p) { return *repoint<bf16x8>(p); }
__device__ __forceinline__ bf16x8 load_row8(const uint16_t* p) { return *repoint<bf16x8>(p); }
template <typename P> __device__ __forceinline__ float8v load_two4(P p) {
  const floatx4 a = ld4f(p), b = ld4f(p + 4);
  return float8v{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ float8v load_row8(const KDA_GLOBAL float* p) { return load_two4(p); }
__device__ __forceinline__ float8v load_row8(const float* p) { return load_two4(p); }

// fragments stored plane by plane (LDS or workspace)
template <typename F> struct FragIo;
template <> struct FragIo<bf16x8> {
  template <typename P> static __device__ __forceinline__ bf16x8 load(P at, int lane) { return *repoint<bf16x8>(at + lane * 16); }
  template <typename P> static __device__ __forceinline__ void store(P at, int lane, bf16x8 f) { *repoint<bf16x8>(at + lane * 16) = f; }
};
template <int N> struct FragIo<Planes<N>> {
  template <typename P> static __device__ __forceinline__ Planes<N> load(P at, int lane) {
    Planes<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) f.p[i] = *repoint<bf16x8>(at + i * kPlane + lane * 16);
    return f;
  }
  template <typename P> static __device__ __forceinline__ void store(P at, int lane, const Planes<N>& f) {
#pragma unroll
    for (int i = 0; i < N; ++i) *repoint<bf16x8>(at + i * kPlane + lane * 16) = f.p[i];
  }
};
template <> struct FragIo<float8v> {
  template <typename P> static __device__ __forceinline__ float8v load(P at, int lane) {
    const floatx4 a = *repoint<floatx4>(at + lane * 16), b = *repoint<floatx4>(at + kPlane + lane * 16);
    return float8v{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  template <typename P> static __device__ __forceinline__ void store(P at, int lane, const float8v& f) {
    *repoint<floatx4>(at + lane * 16) = floatx4{f[0], f[1], f[2], f[3]};
    *repoint<floatx4>(at + kPlane + lane * 16) = floatx4{f[4], f[5], f[6], f[7]};
  }
};
template <typename F, typename P> __device__ __forceinline__ F load_frag(P at, int lane) { return FragIo<F>::load(at, lane); }
template <typename P, typename F> __device__ __forceinline__ void store_frag(P at, int lane, const F& f) { FragIo<F>::store(at, lane, f); }

template <int N> __device__ __forceinline__ Planes<N> make_op(float8v f, uint16_t) {
  Planes<N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bf16x8v h = __builtin_convertvector(f, bf16x8v);
    r.p[i] = __builtin_bit_cast(bf16x8, h);
    f -= __builtin_convertvector(h, float8v);
  }
  return r;
}
template <int N> __device__ __forceinline__ float8v make_op(const float8v& f, float) { return f; }

// A result tile (lane (li, g): rows 4g .. 4g + 3 of column li) as the half `half` (rows 0-15 or 16-31)
// of a fragment's contraction places: 4 consecutive places of one lane, one 8- or 16-byte write a plane
template <int N> __device__ __forceinline__ void put_op(char* frag, int half, int li, int g, floatx4 x, uint16_t) {
  char* at = frag + (li + 16 * (2 * half + (g >> 1))) * 16 + (g & 1) * 8;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t h0 = pk_bf16(x[0], x[1]), h1 = pk_bf16(x[2], x[3]);
    *reinterpret_cast<u32x2v*>(at + i * kPlane) = u32x2v{h0, h1};
    if (i + 1 < N) x -= floatx4{lo_bf16(h0), hi_bf16(h0), lo_bf16(h1), hi_bf16(h1)};
  }
}
template <int N> __device__ __forceinline__ void put_op(char* frag, int half, int li, int g, floatx4 x, float) {
  *reinterpret_cast<floatx4*>(frag + (g & 1) * kPlane + (li + 16 * (2 * half + (g >> 1))) * 16) = x;
}
// A chunk's rows of an input in LDS, and its transpose as an A operand: lane li has channel 16 m + li of 8
// consecutive tokens.  bf16: ds_read_b64_tr_b16, in which 16 lanes read 4 rows of 16 values and get 4 rows of
// one column each; a row length of 8 banks modulo 64 keeps those 4 rows on different banks.
template <typename T, int D> struct Rows {
  static constexpr int kLd = sizeof(T) == 2 ? D + 16 : D + 4;
  T x[64 * kLd];
  // This wavefront's 16 rows from `row0` on: loaded as whole rows (each load covers as few cache lines as it
  // can: a compute unit has only so many requests under way), left here, and read back as the A operand
  // of products over the channels.
  static constexpr int kPieces = D / 8, kLoads = D / 32;   // 16-byte (fp32: 32) pieces of a row, loads a lane
  __device__ __forceinline__ void leave(const typename Frags<T>::In (&v)[kLoads], int row0, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) put8(row0 + (64 * i + lane) / kPieces, (64 * i + lane) % kPieces * 8, v[i]);
  }
  __device__ __forceinline__ typename Frags<T>::In row_frag(int tile, int ks, int lane) const {
    return load_row8(x + (16 * tile + (lane & 15)) * kLd + 32 * ks + 8 * (lane >> 4));
  }
  // row `row`, values c .. c + 7
  __device__ __forceinline__ void put8(int row, int c, const typename Frags<T>::In& v) { *reinterpret_cast<typename Frags<T>::In*>(x + row * kLd + c) = v; }
  __device__ __forceinline__ typename Frags<T>::In transposed(int m, int ks, int lane) const {
    const int li = lane & 15, g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
      typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
      const T* at = x + (32 * ks + 8 * g + (li >> 2)) * kLd + 16 * m + 4 * (li & 3);
      const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_bf16x4*)at);
      const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_bf16x4*)(at + 4 * kLd));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      float8v f;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = x[(32 * ks + 8 * g + e) * kLd + 16 * m + li];
      return f;
    }
  }
};

// one value of a fragment of the inputs' type (its first plane): contraction place `k` of column `col`
template <typename T> __device__ __forceinline__ T frag_at(const char* frag, int k, int col) {
  const int ln = col + 16 * (k >> 3);
  if constexpr (sizeof(T) == 2) return *reinterpret_cast<const T*>(frag + ln * 16 + (k & 7) * 2);
  else return *reinterpret_cast<const T*>(frag + ((k >> 2) & 1) * kPlane + ln * 16 + (k & 3) * 4);
}

// 4 consecutive values of a row in memory (8-byte aligned bf16, 16-byte aligned fp32)
__device__ __forceinline__ floatx4 load_row4(const KDA_GLOBAL uint16_t* p) {
  const u32x2v x = *repoint<u32x2v>(p);
  return floatx4{lo_bf16(x[0]), hi_bf16(x[0]), lo_bf16(x[1]), hi_bf16(x[1])};
}
__device__ __forceinline__ floatx4 load_row4(const KDA_GLOBAL float* p) { return ld4f(p); }
__device__ __forceinline__ void store_row4(KDA_GLOBAL uint16_t* p, floatx4 x) {
  *repoint<u32x2v>(p) = u32x2v{pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3])};
}
__device__ __forceinline__ void store_row4(KDA_GLOBAL float* p, floatx4 x) { *repoint<floatx4>(p) = x; }

// Workgroups of one (sequence, head) read the same operands: they get blocks of one XCD (block b runs
// on XCD b mod 8), so that its L2 serves all but the first.  Returns false for a block without work.
__device__ __forceinline__ bool gdr_block(int64_t block, int64_t units, int parts, int64_t* unit, int* part) {
  const int64_t j = block >> 3;
  *unit = (block & 7) + 8 * (j / parts);
  *part = (int)(j % parts);
  return *unit < units;
}
inline int64_t gdr_blocks(int64_t units, int parts) { return (units + 7) / 8 * 8 * parts; }

}  // namespace kda
