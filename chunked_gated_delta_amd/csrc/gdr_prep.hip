// Per-chunk preparation of the head-gated delta rule: everything that does not depend on the state.
//
// One workgroup of 4 wavefronts per (64-token chunk, key head); wavefront i holds rows 16i .. 16i + 15.
// K K^T and Q K^T are formed once per key head on the matrix cores; per value head that shares it, the
// decay factors D_rj = e^{G_r - G_j} (prefix in double, kept as two floats: differences stay exact
// beside resets of any size) turn them into A and P, and T' = (I + A diag(beta))^{-1} is formed in fp32:
// the four 16 x 16 diagonal blocks by substitution, one a wavefront, then block column j by wavefront j,
//   X_ij = -X_ii sum_{j <= m < i} A_im X_mj,
// on v_mfma_f32_16x16x4_f32, whose result registers are the next product's B operand as they are (the
// contraction runs over places 4g + r).  The backward also needs (I + diag(beta) A)^{-1} and P transposed.
//
// Bound by HBM: it reads K and Q and writes 18 KiB of T' (three planes) and 12 of P (two) a chunk and head; 64K tokens
// of 16 heads take 257 us for 1.05 GB, 4.1 TB/s (a large copy: 4.8), 2 x 4096 tokens' backward 59 us for 0.19 GB.
#include "gdr_internal.h"

namespace kda {

namespace {

constexpr int kLd = 68;   // row length of the 64 x 64 fp32 matrices in LDS

// block column `wave` of (I + N)^{-1}, N strictly lower in mat; the diagonal blocks' inverses go to diag
__device__ __forceinline__ void solve_columns(float* mat, float* diag, int wave, int li, int g, floatx4 (&X)[4]) {
  // column li of the diagonal block's inverse, row by row (every lane group computes the same)
  float x[16];
  const float* blk = mat + 16 * wave * kLd + 16 * wave;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float s = r == li ? 1.f : 0.f;
#pragma unroll
    for (int j = 0; j < r; ++j) s -= blk[r * kLd + j] * x[j];
    x[r] = s;
  }
  float* dg = diag + wave * 16 * 20;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if ((r >> 2) == g) dg[r * 20 + li] = x[r];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) X[i] = floatx4{};
#pragma unroll
  for (int j = 0; j < 4; ++j)   // X_jj, j = wave
    if (j == wave) {
#pragma unroll
      for (int r = 0; r < 4; ++r) X[j][r] = diag[j * 320 + (4 * g + r) * 20 + li];
    }
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    if (i <= wave) continue;
    floatx4 acc = {};
#pragma unroll
    for (int m = 0; m < i; ++m) {
      if (m < wave) continue;
      const floatx4 a = ld4f(mat + (16 * i + li) * kLd + 16 * m + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], X[m][r], acc, 0, 0, 0);
    }
    const floatx4 d = ld4f(diag + i * 320 + li * 20 + 4 * g);
    floatx4 out = {};
#pragma unroll
    for (int r = 0; r < 4; ++r) out = __builtin_amdgcn_mfma_f32_16x16x4f32(-d[r], acc[r], out, 0, 0, 0);
    X[i] = out;
  }
}

// fragments of a matrix in LDS as an A operand: lane holds 8 consecutive columns of row li of the tile
__device__ __forceinline__ float8v rows_frag(const float* mat, int tile, int ks, int li, int g) {
  return load_row8(mat + (16 * tile + li) * kLd + 32 * ks + 8 * g);
}
// the same of its transpose
__device__ __forceinline__ float8v cols_frag(const float* mat, int tile, int ks, int li, int g) {
  float8v f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = mat[(32 * ks + 8 * g + e) * kLd + 16 * tile + li];
  return f;
}

template <typename T, int DK, bool BWD>
__global__ __launch_bounds__(256) void gdr_prep_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  constexpr int KS = DK / 32;
  constexpr int kInFrag = in_frag<T>(), kOpFrag = op_frag<T, 3>();
  __shared__ __attribute__((aligned(16))) char kf[4 * KS * kInFrag];   // a row operand's fragments [tile][step]
  __shared__ __attribute__((aligned(16))) float mat[64 * kLd];
  __shared__ __attribute__((aligned(16))) float diag[4 * 320];
  __shared__ float ghi[64], glo[64], bet[64];

  const int64_t slot = blockIdx.x;
  const int kh = blockIdx.y;
  GdrSeq seq;
  int64_t chunk;
  if (!gdr_find(p, slot, &seq, &chunk)) return;
  const int lane = threadIdx.x & 63, wave = wave_id(), li = lane & 15, g = lane >> 4;
  const int64_t t0 = seq.t0 + chunk * kGdrChunk;
  const int64_t left = seq.len - chunk * kGdrChunk;
  const int n = left < kGdrChunk ? (int)left : kGdrChunk;   // tokens of this chunk

  // this wavefront's rows of K and Q
  In kr[KS], qr[KS];
  {
    const int row = 16 * wave + li;
    const auto kp = global_in<T>(p.k) + seq.row * p.sk.b + kh * p.sk.h + (t0 + row) * p.sk.t + 8 * g;
    const auto qp = global_in<T>(p.q) + seq.row * p.sq.b + kh * p.sq.h + (t0 + row) * p.sq.t + 8 * g;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      zero_frag(kr[ks]);
      zero_frag(qr[ks]);
      if (row < n) {
        kr[ks] = load_row8(kp + 32 * ks);
        qr[ks] = load_row8(qp + 32 * ks);
      }
    }
  }
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) store_frag(kf + (wave * KS + ks) * kInFrag, lane, kr[ks]);
  __syncthreads();

  floatx4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = floatx4{};
    qk[j] = floatx4{};
    if (j > wave) continue;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const In b = load_frag<In>(kf + (j * KS + ks) * kInFrag, lane);
      kk[j] = mma(kr[ks], b, kk[j]);
      qk[j] = mma(qr[ks], b, qk[j]);
    }
  }

  const int grp = p.Hv / p.Hk;
  for (int hg = 0; hg < grp; ++hg) {
    const int h = kh * grp + hg;
    const int64_t blk = slot * p.Hv + h;
    const auto gate = global_out<float>(p.ws_gate) + blk * kGateFloats;
    if (wave == 0) {   // one token a lane
      double G = 0.0;
      float b = 0.f;
      if (lane < n) {
        G = (double)gdr_gate(get(global_in<T>(p.w) + seq.row * p.sw.b + h * p.sw.h + (t0 + lane) * p.sw.t), p.gate, p.g_min);
        b = get(global_in<T>(p.beta) + seq.row * p.sb.b + h * p.sb.h + (t0 + lane) * p.sb.t);
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double up = __shfl_up(G, d);
        if (lane >= d) G += up;
      }
      const double last = __shfl(G, 63);
      const float hi = (float)G, lo = (float)(G - (double)hi);
      ghi[lane] = hi;
      glo[lane] = lo;
      bet[lane] = b;
      gate[kGateGam + lane] = expf(hi) * (1.f + lo);
      gate[kGateEta + lane] = expf((float)(last - G));
      gate[kGateBeta + lane] = b;
      gate[kGateHi + lane] = hi;
      gate[kGateLo + lane] = lo;
      if (lane == 0) gate[kGateLast] = expf((float)last);
    }
    __syncthreads();
    floatx4 D[4] = {}, X[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > wave) continue;
      const int col = 16 * j + li;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * wave + 4 * g + r;
        D[j][r] = row >= col ? expf((ghi[row] - ghi[col]) + (glo[row] - glo[col])) : 0.f;
      }
    }
    constexpr int kVariants = BWD ? 2 : 1;
#pragma unroll
    for (int variant = 0; variant < kVariants; ++variant) {
      // N = A diag(beta), or diag(beta) A for the adjoint
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * wave + 4 * g + r, col = 16 * j + li;
          mat[row * kLd + col] = row > col ? kk[j][r] * D[j][r] * bet[variant ? row : col] : 0.f;
        }
      }
      __syncthreads();
      solve_columns(mat, diag, wave, li, g, X);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) mat[(16 * i + 4 * g + r) * kLd + 16 * wave + li] = X[i][r];
      __syncthreads();
      if (variant == 0) {
        const auto out = as_global(p.ws_ti) + blk * kTriFrags * kOpFrag;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks <= wave / 2) store_frag(out + lower_frag(wave, ks) * kOpFrag, lane, make_op<3>(rows_frag(mat, wave, ks, li, g), T{}));
      } else {
        const auto out = as_global(p.ws_tt) + blk * kTriFrags * kOpFrag;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks >= wave / 2) store_frag(out + upper_frag(wave, ks) * kOpFrag, lane, make_op<3>(cols_frag(mat, wave, ks, li, g), T{}));
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * wave + 4 * g + r, col = 16 * j + li;
        mat[row * kLd + col] = row >= col ? p.scale * qk[j][r] * D[j][r] : 0.f;
      }
    __syncthreads();
    if constexpr (BWD) {
      const auto out = as_global(p.ws_p) + blk * kTriFrags * kOpFrag;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks >= wave / 2) store_frag(out + upper_frag(wave, ks) * kOpFrag, lane, make_op<3>(cols_frag(mat, wave, ks, li, g), T{}));
    } else {
      // the outputs' own factor, two planes: one, as coarse as o itself, raises o's error from 1.7e-3 to 2.3e-3
      const auto out = as_global(p.ws_p) + blk * kTriFrags * op_frag<T, 2>();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks <= wave / 2) store_frag(out + lower_frag(wave, ks) * op_frag<T, 2>(), lane, make_op<2>(rows_frag(mat, wave, ks, li, g), T{}));
    }
    __syncthreads();
  }
}

template <typename T, bool BWD>
hipError_t launch_t(const GdrParams& p, hipStream_t s) {
  const int64_t slots = gdr_slots(p.B, p.T, p.n_seq, p.seq_start != nullptr);
  if (slots == 0) return hipSuccess;
  const dim3 grid((unsigned)slots, (unsigned)p.Hk);
  switch (p.dk) {
    case 32: hipLaunchKernelGGL((gdr_prep_kernel<T, 32, BWD>), grid, dim3(256), 0, s, p); break;
    case 64: hipLaunchKernelGGL((gdr_prep_kernel<T, 64, BWD>), grid, dim3(256), 0, s, p); break;
    default: hipLaunchKernelGGL((gdr_prep_kernel<T, 128, BWD>), grid, dim3(256), 0, s, p); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_prep(const GdrParams& p, hipStream_t s, bool bwd) {
  if (p.dtype == KDA_DTYPE_BF16) return bwd ? launch_t<uint16_t, true>(p, s) : launch_t<uint16_t, false>(p, s);
  return bwd ? launch_t<float, true>(p, s) : launch_t<float, false>(p, s);
}

}  // namespace kda
