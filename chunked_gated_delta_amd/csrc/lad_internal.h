// Internal declarations of linear attention with a decay for each head.
//
// One walk does everything: with a state S (DX x DZ) and rows X, Y (DX values) and Z (DZ values),
//     S <- e^{g_t} S + Y_t Z_t^T;   out_t = S^T X_t
// is the forward with (X, Y, Z) = (q, k, v) and gives dq with (dO, v, k); backwards in time, with the
// decay taken behind the output, it gives dk with (v, dO, q) and dv with (k, q, dO).  In chunks of C = 64 tokens
// in the walk's order, P the prefix of the log-decays in the chunk (inclusive forwards, exclusive backwards):
//     out_i = e^{P_i} X_i S + sum_{j <= i} e^{P_i - P_j} (X_i . Y_j) Z_j
//     S <- e^{Ptot} S + sum_j e^{Ptot - P_j} Y_j Z_j^T
// Every exponent is at most 0, and one decay a head keeps it out of the bf16 operands of X Y^T.
//
// Long sequences are cut into segments of L tokens that walk side by side: a first launch forms each segment's
// state from zero, a second chains them (S entering segment i + 1 = e^{decay of i} S entering i + that state).
#pragma once

#include "gdr_internal.h"

namespace kda {

struct LadWalk {
  const void *x, *y, *z, *dot;              // rows; dot nullable
  kda_stride_t sx, sy, sz, sdot;
  int grp_x, grp_y, grp_z, grp_dot;         // value heads that share a head of the tensor
  void* out;
  kda_stride_t so;
  const float* entering;                    // per (slot, head) with by_slot, else per (sequence, head); null: zero
  float* leaving;                           // per (slot, head) with leave_slot, else per (sequence, head), behind the walk's last segment; nullable
  float* decay;                             // e^{the segment's decay} per (slot, head); nullable
  double* dots[2];                          // [B, Hv, T]: out_t . dot_t of what came from the state, and of all of it
  float out_scale, in_scale;                // of the outputs, and of Z in outputs and state
  int reverse, transposed, by_slot, leave_slot, out_f32, skip_end;   // transposed: states lie as [DZ][DX]; skip_end: no walk over the segment
                                                         // behind which none comes
};

struct LadParams {
  LadWalk walk[3];
  int n_walks;
  const void* w;
  kda_stride_t sw;
  int w_per_head, gate;
  float g_min;
  const int32_t* seq_start;                 // packed sequences: n_seq + 1 offsets; null: every batch row is one
  int64_t T, L, n_seq, slots;
  int Hv, grp;
};

// chains the segments' states: S (forwards) and its adjoint R (backwards)
struct LadScan {
  float *s, *r;                             // per (slot, head): in: the segment's own state; out: the one entering it (r: from behind)
  const float *s_decay, *r_decay;
  const float *S0, *dSf;                    // nullable
  float *S_final, *dS0;                     // per (sequence, head); nullable
  const int32_t* seq_start;
  int64_t T, L, n_seq;
  int Hv, size, dirs;                       // size = dk dv; 1: forwards, 2: its adjoint too
};

// the log-decay's gradient from dots of q.dq and k.dk
struct LadDecayGrad {
  const double *qdq[2], *kdk[2];            // [B, Hv, T]: from other chunks, and all
  const float *s, *r;                       // entering states of the segments, where sequences have several
  const float *S0, *S_final, *dSf, *dS0;    // per (sequence, head); S0, dSf nullable; S_final with dSf, dS0 with S0
  const void* w;
  kda_stride_t sw, sdw;
  void* dw;
  double* partial;                          // per (slot, head), of w per head
  const int32_t* seq_start;
  int64_t T, L, n_seq, slots;
  int Hv, size, w_per_head, gate, dtype;
  float g_min;
};

// dq or dk from the value heads that share it
struct LadSum {
  const float* part[2];                     // [B, Hk, grp, T, D]
  void* out[2];                             // dq, dk
  kda_stride_t so[2];
  const int32_t* seq_start;
  int64_t B, T, n_seq;
  int Hk, grp, D, dtype;
};

struct LadStepParams {
  const void *q, *k, *v, *w;
  kda_stride_t sq, sk, sv, sw, so;
  const int32_t* slots;
  float* S;
  void* o;
  int64_t B, T, n_slots;
  int Hk, Hv, dk, dv;
  int dtype, gate, w_per_head;
  float g_min, scale;
};

struct QkNormParams {
  const void *x[2], *weight[2], *dy[2];     // queries, keys
  void *y[2], *dx[2], *dweight[2];
  kda_stride_t sx[2], sy[2], sdy[2], sdx[2];
  const void* positions;
  const float* inv_freq;
  int64_t pos_b, pos_t, B, T;
  int H[2], D, R, dtype, wdtype, norm, interleaved, wide;
  float scale[2], eps;
  float* partial;
};

// chunks of a segment at most: what launch_lad_decay_grad keeps of them fits LDS
constexpr int64_t kLadMaxChunks = 1024;
// segment length, and the number of slots that segments of it need
int64_t lad_segment(const kda_lad_t* d, bool bwd);
int64_t lad_slots(int64_t B, int64_t T, int64_t n_seq, int64_t L, bool packed);

// the walks of p over every segment; states: only their states (no outputs)
hipError_t launch_lad_fwd(const LadParams& p, int dtype, int dx, int dz, hipStream_t s);
// three walks: dq, dk (over dx, dz) and dv (over dz, dx); exact: with fp32's accuracy up to the results' own rounding
hipError_t launch_lad_bwd(const LadParams& p, int dtype, int dx, int dz, bool exact, hipStream_t s);
hipError_t launch_lad_bwd_exact(const LadParams& p, int dtype, int dx, int dz, hipStream_t s);
hipError_t launch_lad_states(const LadParams& p, int dtype, int dx, int dz, hipStream_t s);
hipError_t launch_lad_scan(const LadScan& p, hipStream_t s);
hipError_t launch_lad_decay_grad(const LadDecayGrad& p, hipStream_t s);
hipError_t launch_lad_sum(const LadSum& p, hipStream_t s);
hipError_t launch_lad_step(const LadStepParams& p, hipStream_t s);
size_t qk_norm_bwd_workspace_bytes(const QkNormParams& p);
hipError_t launch_qk_norm_fwd(const QkNormParams& p, hipStream_t s);
hipError_t launch_qk_norm_bwd(const QkNormParams& p, hipStream_t s);

// ---------------------------------------------------------------- segments

struct LadSeg {
  int64_t seq, row, t0, len, seg, n_seg, slot0;   // sequence, batch row, its first token, its tokens; segment of it, segments, first slot
};

// A sequence of len tokens has max(1, ceil(len / L)) segments; packed ones keep them at slot floor(start / L) +
// sequence, which leaves room for every sequence's last one without a prefix sum over the lengths.  Offsets are
// clamped into [0, T], so that offsets out of order address nothing out of range.  T, L < 2^31 and slots < 2^24 (checked on
// the host), so 32 bits divide them: a 64-bit division is 130 instructions in front of everything.
__device__ __forceinline__ LadSeg lad_seq(const int32_t* seq_start, int64_t T, int64_t L, int64_t s) {
  LadSeg q;
  q.seq = s;
  q.seg = 0;
  const uint32_t L_ = (uint32_t)L;
  if (!seq_start) {
    q.row = s;
    q.t0 = 0;
    q.len = T;
    q.n_seg = T > L ? ((uint32_t)T + L_ - 1) / L_ : 1;
    q.slot0 = s * q.n_seg;
  } else {
    const int64_t a = clamp_off(seq_start[s], 0, T), e = clamp_off(seq_start[s + 1], a, T);
    q.row = 0;
    q.t0 = a;
    q.len = e - a;
    q.n_seg = q.len > L ? ((uint32_t)q.len + L_ - 1) / L_ : 1;
    q.slot0 = (uint32_t)a / L_ + s;
  }
  return q;
}

// the segment at this slot; false where the slot holds none
__device__ __forceinline__ bool lad_find(const int32_t* seq_start, int64_t T, int64_t L, int64_t n_seq, int64_t slot, LadSeg* out) {
  int64_t lo = 0;
  const uint32_t L_ = (uint32_t)L;
  if (!seq_start) {
    lo = (uint32_t)slot / (T > L ? ((uint32_t)T + L_ - 1) / L_ : 1u);
  } else {
    int64_t hi = n_seq - 1;   // the last sequence whose first slot is not behind this one
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) / 2;
      if ((uint32_t)clamp_off(seq_start[mid], 0, T) / L_ + mid <= slot) lo = mid; else hi = mid - 1;
    }
  }
  *out = lad_seq(seq_start, T, L, lo);
  out->seg = slot - out->slot0;
  return out->seg >= 0 && out->seg < out->n_seg;
}

// log-decay of one token
template <typename T>
__device__ __forceinline__ float lad_decay(const void* w, int per_head, kda_stride_t sw, int64_t row, int h, int64_t t, int gate, float g_min) {
  const float x = per_head ? global_in<float>(w)[h] : get(global_in<T>(w) + row * sw.b + h * sw.h + t * sw.t);
  return gdr_gate(x, gate, g_min);
}

// ---------------------------------------------------------------- sums over a wavefront

// A value of a lane before (DPP control CTRL, into the rows of ROWS), 0 where there is none
template <int CTRL, int ROWS> __device__ __forceinline__ float behind_lane(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS> __device__ __forceinline__ double behind_lane(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)lo | ((uint64_t)(uint32_t)hi << 32));
}
// sum over the lanes up to this one
template <typename F> __device__ __forceinline__ F lane_prefix(F p) {
  p += behind_lane<0x111, 0xf>(p);   // 1, 2, 4, 8 lanes before, in rows of 16
  p += behind_lane<0x112, 0xf>(p);
  p += behind_lane<0x114, 0xf>(p);
  p += behind_lane<0x118, 0xf>(p);
  p += behind_lane<0x142, 0xa>(p);   // the last lane of rows 0 and 2 to rows 1 and 3
  p += behind_lane<0x143, 0xc>(p);   // lane 31 to rows 2 and 3
  return p;
}
// the last lane's value
__device__ __forceinline__ float last_lane(float x) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63)); }
__device__ __forceinline__ double last_lane(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63) |
                                        ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), 63) << 32));
}
template <typename F> __device__ __forceinline__ F lane_sum(F x) { return last_lane(lane_prefix(x)); }

}  // namespace kda
