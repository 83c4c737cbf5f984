// Host side of linear attention with a decay for each head: argument validation (before any HIP call), segments,
// workspace layout, launches.
#include <cmath>

#include "host_checks.h"
#include "lad_internal.h"

namespace {

using namespace kda;

// sizes, types and the gate
int check_lad(const kda_lad_t* d, bool packed) {
  if (!d) return KDA_ERR_NULL;
  if (d->B < 1 || d->Hk < 1 || d->Hv < 1 || d->T < 0 || d->dk < 1 || d->dv < 1) return KDA_ERR_SHAPE;
  if (d->Hk > 65535 || d->Hv > 65535 || d->Hv % d->Hk != 0) return KDA_ERR_SHAPE;
  if (d->T > 0x7fffffffll || d->B > 0x7fffffffll) return KDA_ERR_SHAPE;
  if (packed ? (d->B != 1 || d->n_seq < 1 || d->n_seq > 0x7fffffffll) : d->n_seq != 0) return KDA_ERR_SHAPE;
  if (!head_dim(d->dk) || !head_dim(d->dv)) return KDA_ERR_UNSUPPORTED;
  if (d->dtype != KDA_DTYPE_F32 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
  if (d->gate != KDA_GATE_BOUNDED && d->gate != KDA_GATE_SOFTPLUS && d->gate != KDA_GATE_LOG) return KDA_ERR_UNSUPPORTED;
  if (d->w_per_head != 0 && d->w_per_head != 1) return KDA_ERR_ARG;
  if (d->gate == KDA_GATE_BOUNDED && !(d->g_min <= 0.f && std::isfinite(d->g_min))) return KDA_ERR_ARG;
  if (!std::isfinite(d->scale)) return KDA_ERR_ARG;
  // a grid holds fewer than 2^24 workgroups of 256 threads (the step: one for 32 value columns)
  const int64_t n_seq = packed ? d->n_seq : d->B;
  if ((double)n_seq * d->Hv * (d->dv / 32) >= (double)(1 << 23)) return KDA_ERR_SHAPE;
  if ((double)d->B * d->T * d->Hv * 4.0 > (double)kMaxExtent) return KDA_ERR_SHAPE;
  return KDA_OK;
}

struct Plan {
  int64_t n_seq, L, slots;
  int grp;
};

Plan plan_of(const kda_lad_t* d, bool packed, bool bwd) {
  Plan p;
  p.n_seq = packed ? d->n_seq : d->B;
  p.grp = (int)(d->Hv / d->Hk);
  p.L = lad_segment(d, bwd);
  p.slots = lad_slots(d->B, d->T, p.n_seq, p.L, packed);
  return p;
}

// and the launches of the chunked kernels: the walks (three, blocks of 8 units), the chain over 1024 values of a state
int check_chunked(const kda_lad_t* d, bool packed, bool bwd) {
  const int rc = check_lad(d, packed);
  if (rc != KDA_OK) return rc;
  const Plan p = plan_of(d, packed, bwd);
  const double most = (double)(1 << 24);
  if (((double)p.slots * (double)d->Hk + 8) * p.grp * 3 >= most) return KDA_ERR_SHAPE;
  if ((double)p.n_seq * (double)d->Hv * 2 * (double)((d->dk * d->dv + 1023) / 1024) >= most) return KDA_ERR_SHAPE;
  if ((double)p.slots * (double)d->Hv * (double)(d->dk * d->dv) * 4.0 > (double)kMaxExtent) return KDA_ERR_SHAPE;
  return KDA_OK;
}

int check_inputs(const kda_lad_t* d, const void* q, const void* k, const void* v, const void* w) {
  const int64_t B = d->B, T = d->T, e = elem(d->dtype);
  if (T > 0 && (!q || !k || !v || !w)) return KDA_ERR_NULL;
  int rc;
  if ((rc = check_strides(q, d->q, B, d->Hk, T, d->dk, e, 16)) != KDA_OK) return rc;
  if ((rc = check_strides(k, d->k, B, d->Hk, T, d->dk, e, 16)) != KDA_OK) return rc;
  if ((rc = check_strides(v, d->v, B, d->Hv, T, d->dv, e, 16)) != KDA_OK) return rc;
  if (d->w_per_head) return aligned(w, 4) ? KDA_OK : KDA_ERR_ARG;
  return check_strides(w, d->w, B, d->Hv, T, 1, e, e);
}

Span w_span(const kda_lad_t* d, const void* w) {
  return d->w_per_head ? dense(w, d->Hv * 4.0) : view(w, d->w, d->B, d->Hv, d->T, 1, elem(d->dtype));
}

// workspace sections
struct Work {
  char *s, *r, *s_decay, *r_decay, *s_final, *r_start;   // the chain over the segments, and what leaves it
  char *qdq, *kdk, *partial;                   // of the decay's gradient; qdq and kdk twice [B, Hv, T]
  char *dq, *dk;                               // gradients by value head, where heads share q and k
};

size_t layout(Work& w, void* base, const kda_lad_t* d, const Plan& p, bool bwd) {
  size_t off = 0;
  auto take = [&](char*& at, double bytes) {
    at = base ? static_cast<char*>(base) + off : nullptr;
    off += ((size_t)bytes + 255) / 256 * 256;
  };
  const double per_slot = (double)p.slots * d->Hv, size = (double)d->dk * d->dv * 4, rows = (double)d->B * d->Hv * d->T * 4;
  w = Work{};
  if (bwd || d->T > p.L) {
    take(w.s, per_slot * size);
    take(w.s_decay, per_slot * 4);
  }
  if (!bwd) return off;
  take(w.r, per_slot * size);
  take(w.r_decay, per_slot * 4);
  take(w.s_final, (double)p.n_seq * d->Hv * size);
  take(w.r_start, (double)p.n_seq * d->Hv * size);
  take(w.qdq, rows * 4);   // two of doubles
  take(w.kdk, rows * 4);
  take(w.partial, per_slot * 8);
  if (p.grp > 1) {
    take(w.dq, rows * d->dk);
    take(w.dk, rows * d->dk);
  }
  return off;
}

LadParams params(const kda_lad_t* d, const Plan& pl, const void* w, const int32_t* seq_start) {
  LadParams p{};
  p.w = w; p.sw = d->w; p.w_per_head = d->w_per_head; p.gate = d->gate; p.g_min = d->g_min;
  p.seq_start = seq_start; p.T = d->T; p.L = pl.L; p.n_seq = pl.n_seq; p.slots = pl.slots;
  p.Hv = (int)d->Hv; p.grp = pl.grp;
  return p;
}

struct Tensor {
  const void* p;
  kda_stride_t s;
  int grp;
};

LadWalk walk_over(Tensor x, Tensor y, Tensor z) {
  LadWalk k{};
  k.x = x.p; k.sx = x.s; k.grp_x = x.grp;
  k.y = y.p; k.sy = y.s; k.grp_y = y.grp;
  k.z = z.p; k.sz = z.s; k.grp_z = z.grp;
  k.grp_dot = 1;
  k.out_scale = k.in_scale = 1.f;
  return k;
}

float* floats(char* p) { return reinterpret_cast<float*>(p); }

}  // namespace

namespace kda {

// Tokens of a segment.  Up to 3 chunks are not worth three launches.  Otherwise n segments and heads at a time:
//  - as many as workgroups run at once: two a compute unit, one of fp32 with a side of 128; the gradients' three walks
//    take a third each, or half where their workgroups are small or long (fp32);
//  - a chunk of a segment is some a us of a walk and of its state's (less with more segments), a segment's state some b us of
//    the memory's time: n^2 = a / b times the chunks.  With decays of at most 0.02 a token, so that no head forgets early, two
//    sequences of 2048 tokens, 16 heads of 128 x 128, bf16: 8, 11 (this rule) and 32 segments a head's forward 53, 56 and 81 us; of
//    4096 tokens 8, 16 (this rule) and 32 79, 77 and 102; 64K tokens of one with 32 (this rule) 409, with 16 461; gradients of
//    2 x 4096 with 5 (this rule) 178 us, with 4 194, 8 173, 11 197.  9 packed prompts, 4099 tokens, 16 heads: 30 segments a head
//    62 us, 21 69, 41 75.  Within 5 % of the best of each sweep;
//  - the chain over a sequence's segments is serial: c chunks each at least, c^2 = T / 1250.
// The gradients' segments have at most 16 chunks where the chain allows it, also where fewer would fill the machine: the
// decay's gradient starts from <S, R> at their ends, and carried over more than that it takes rounding from far away
// (lad_decay_grad_kernel).  16 x 4096 tokens, 16 heads of 128 x 128, bf16, in one segment a row and in four: 928 and 973 us where
// decays forget, 934 and 1178 where they keep everything; with dS0, which a single segment's walks leave in three planes, 1501
// and 971.
int64_t lad_segment(const kda_lad_t* d, bool bwd) {
  const int64_t T = d->T;
  if (T <= 3 * kGdrChunk) return 3 * kGdrChunk;
  const double chunks = (double)d->B * (double)T * (double)d->Hv / kGdrChunk, state = (double)(d->dk * d->dv) / 16384.0;
  const bool f32 = d->dtype == KDA_DTYPE_F32, wide = d->dk == 128 || d->dv == 128;
  const double capacity = bwd ? (wide && !f32 ? 170.0 : 256.0) : (wide && f32 ? 256.0 : 512.0);
  const double fair = std::sqrt((bwd ? 70.0 : d->n_seq > 0 ? 200.0 : 120.0) * chunks / state);
  const int64_t at_once = (int64_t)((fair < capacity ? fair : capacity) / (double)d->Hv);   // segments of a head
  int64_t n;
  if (d->n_seq > 0) n = at_once > d->n_seq ? at_once - d->n_seq / 2 : at_once / 2;   // their last ones are partly filled
  else n = at_once / d->B;
  int64_t L = n > 0 ? (T + n - 1) / n : T;
  int64_t least = kGdrChunk * (int64_t)(0.5 + std::sqrt((double)T / 1250.0));
  if (bwd && least > kGdrChunk * kLadMaxChunks) least = kGdrChunk * kLadMaxChunks;
  const int64_t most = kGdrChunk * 16;
  if (bwd && L > most) L = most;
  if (L < least) L = least;
  return (L + kGdrChunk - 1) / kGdrChunk * kGdrChunk;
}

int64_t lad_slots(int64_t B, int64_t T, int64_t n_seq, int64_t L, bool packed) {
  return packed ? T / L + n_seq : B * (T > L ? (T + L - 1) / L : 1);
}

}  // namespace kda

extern "C" {

size_t kda_lad_workspace_bytes(const kda_lad_t* desc, int backward) {
  if (!desc || check_chunked(desc, desc->n_seq != 0, backward != 0) != KDA_OK) return (size_t)-1;
  Work w;
  return layout(w, nullptr, desc, plan_of(desc, desc->n_seq != 0, backward != 0), backward != 0);
}

int kda_lad_chunk_fwd(const void* q, const void* k, const void* v, const void* w, const float* S0, const int32_t* seq_start,
                      const kda_lad_t* desc, void* o, const kda_stride_t* o_stride, float* S_final, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int rc = check_chunked(desc, seq_start != nullptr, false);
  if (rc != KDA_OK) return rc;
  const int64_t B = desc->B, Hk = desc->Hk, Hv = desc->Hv, T = desc->T, dk = desc->dk, dv = desc->dv, e = elem(desc->dtype);
  if ((rc = check_inputs(desc, q, k, v, w)) != KDA_OK) return rc;
  if (T > 0 && (!o || !o_stride)) return KDA_ERR_NULL;
  const kda_stride_t so = o_stride ? *o_stride : kda_stride_t{};
  if ((rc = check_out(o, so, B, Hv, T, dv, e, 16)) != KDA_OK) return rc;
  if (!aligned(S0, 16) || !aligned(S_final, 16) || !aligned(workspace, 16) || !aligned(seq_start, 4)) return KDA_ERR_ARG;
  const Plan pl = plan_of(desc, seq_start != nullptr, false);
  Work ws;
  const size_t need = layout(ws, workspace, desc, pl, false);
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_ARG;
  const double states = (double)pl.n_seq * Hv * dk * dv * 4;
  const Span s0 = dense(S0, states), sf = dense(S_final, states), out = view(o, so, B, Hv, T, dv, e), wsp = dense(workspace, (double)need);
  const Span start = dense(seq_start, seq_start ? (desc->n_seq + 1) * 4.0 : 0);
  if ((rc = check_apart({view(q, desc->q, B, Hk, T, dk, e), view(k, desc->k, B, Hk, T, dk, e), view(v, desc->v, B, Hv, T, dv, e),
                         w_span(desc, w), start},
                        {out, sf, wsp})) != KDA_OK)
    return rc;
  if (meet(s0, out) || meet(s0, wsp) || (S0 != S_final && meet(s0, sf))) return KDA_ERR_ARG;   // S_final may be S0
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  LadParams p = params(desc, pl, w, seq_start);
  p.n_walks = 1;
  LadWalk& k0 = p.walk[0];
  const Tensor rk{k, desc->k, pl.grp}, rv{v, desc->v, 1};
  if (need > 0) {
    k0 = walk_over({}, rk, rv);
    k0.grp_x = 1;
    k0.leaving = floats(ws.s);
    k0.leave_slot = 1;
    k0.decay = floats(ws.s_decay);
    k0.skip_end = !S_final;
    if ((rc = done(launch_lad_states(p, desc->dtype, (int)dk, (int)dv, s))) != KDA_OK) return rc;
    LadScan sc{};
    sc.s = floats(ws.s); sc.s_decay = floats(ws.s_decay); sc.S0 = S0; sc.S_final = S_final; sc.seq_start = seq_start;
    sc.T = T; sc.L = pl.L; sc.n_seq = pl.n_seq; sc.Hv = (int)Hv; sc.size = (int)(dk * dv); sc.dirs = 1;
    if ((rc = done(launch_lad_scan(sc, s))) != KDA_OK) return rc;
  }
  k0 = walk_over({q, desc->q, pl.grp}, rk, rv);
  k0.out = o;
  k0.so = so;
  k0.out_scale = desc->scale;
  k0.entering = need > 0 ? floats(ws.s) : S0;
  k0.by_slot = need > 0;
  k0.leaving = need > 0 ? nullptr : S_final;
  return done(launch_lad_fwd(p, desc->dtype, (int)dk, (int)dv, s));
}

int kda_lad_chunk_bwd(const void* q, const void* k, const void* v, const void* w, const float* S0, const int32_t* seq_start,
                      const kda_lad_t* desc, const void* dO, const kda_stride_t* dO_stride, const float* dS_final,
                      const kda_lad_grads_t* grads, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_chunked(desc, seq_start != nullptr, true);
  if (rc != KDA_OK) return rc;
  if (!grads) return KDA_ERR_NULL;
  const int64_t B = desc->B, Hk = desc->Hk, Hv = desc->Hv, T = desc->T, dk = desc->dk, dv = desc->dv, e = elem(desc->dtype);
  if ((rc = check_inputs(desc, q, k, v, w)) != KDA_OK) return rc;
  if (T > 0 && (!dO || !dO_stride || !grads->dq || !grads->dk || !grads->dv)) return KDA_ERR_NULL;
  const kda_stride_t sdo = dO_stride ? *dO_stride : kda_stride_t{};
  if ((rc = check_strides(dO, sdo, B, Hv, T, dv, e, 16)) != KDA_OK) return rc;
  if ((rc = check_out(grads->dq, grads->sq, B, Hk, T, dk, e, 16)) != KDA_OK) return rc;
  if ((rc = check_out(grads->dk, grads->sk, B, Hk, T, dk, e, 16)) != KDA_OK) return rc;
  if ((rc = check_out(grads->dv, grads->sv, B, Hv, T, dv, e, 16)) != KDA_OK) return rc;
  const bool per_head = desc->w_per_head != 0;
  if (per_head && grads->dw && (!aligned(grads->dw, 4) || !w)) return w ? KDA_ERR_ARG : KDA_ERR_NULL;
  if (!per_head && (rc = check_out(grads->dw, grads->sw, B, Hv, T, 1, e, e)) != KDA_OK) return rc;
  if (!aligned(S0, 16) || !aligned(dS_final, 16) || !aligned(grads->dS0, 16) || !aligned(workspace, 16) || !aligned(seq_start, 4))
    return KDA_ERR_ARG;
  const Plan pl = plan_of(desc, seq_start != nullptr, true);
  Work ws;
  const size_t need = layout(ws, workspace, desc, pl, true);
  if (!workspace || workspace_bytes < need) return KDA_ERR_ARG;
  const double states = (double)pl.n_seq * Hv * dk * dv * 4;
  if ((rc = check_apart({view(q, desc->q, B, Hk, T, dk, e), view(k, desc->k, B, Hk, T, dk, e), view(v, desc->v, B, Hv, T, dv, e),
                         w_span(desc, w), dense(seq_start, seq_start ? (desc->n_seq + 1) * 4.0 : 0), view(dO, sdo, B, Hv, T, dv, e),
                         dense(S0, states), dense(dS_final, states)},
                        {view(grads->dq, grads->sq, B, Hk, T, dk, e), view(grads->dk, grads->sk, B, Hk, T, dk, e),
                         view(grads->dv, grads->sv, B, Hv, T, dv, e),
                         per_head ? dense(grads->dw, Hv * 4.0) : view(grads->dw, grads->sw, B, Hv, T, 1, e),
                         dense(grads->dS0, states), dense(workspace, (double)need)})) != KDA_OK)
    return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  LadParams p = params(desc, pl, w, seq_start);
  const Tensor rq{q, desc->q, pl.grp}, rk{k, desc->k, pl.grp}, rv{v, desc->v, 1}, rdo{dO, sdo, 1};
  // Sequences of several segments have their states formed and chained first.  A single segment's walks take the entering
  // states as they are given and leave S behind the last token and dS0 themselves, in three planes, for two launches less
  // (64 tokens of 4 heads: 34 -> 25 us).  Many short rows pay for the planes: 16 heads of 128 x 128 in bf16, without dS0 and with
  // it, 16 x 64 tokens 28 and 46 us, 64 x 192 tokens 184 and 339, 512 x 64 tokens 550 and 1115.
  const bool segments = T > pl.L;
  // <S, R> behind the last token and in front of the first
  const bool want_end = dS_final && grads->dw, want_start = S0 && grads->dw;
  float* const r_start = grads->dS0 ? grads->dS0 : want_start ? floats(ws.r_start) : nullptr;
  if (segments) {
    p.n_walks = 2;
    LadWalk &f = p.walk[0], &r = p.walk[1];
    f = walk_over({nullptr, {}, 1}, rk, rv);
    f.leaving = floats(ws.s); f.leave_slot = 1; f.decay = floats(ws.s_decay); f.skip_end = !want_end;
    r = walk_over({nullptr, {}, 1}, rq, rdo);
    r.leaving = floats(ws.r); r.leave_slot = 1; r.decay = floats(ws.r_decay); r.skip_end = !r_start;
    r.reverse = 1;
    r.in_scale = desc->scale;
    if ((rc = done(launch_lad_states(p, desc->dtype, (int)dk, (int)dv, s))) != KDA_OK) return rc;
    LadScan sc{};
    sc.s = floats(ws.s); sc.s_decay = floats(ws.s_decay); sc.S0 = S0; sc.S_final = want_end ? floats(ws.s_final) : nullptr;
    sc.r = floats(ws.r); sc.r_decay = floats(ws.r_decay); sc.dSf = dS_final; sc.dS0 = r_start;
    sc.dirs = 2;
    sc.seq_start = seq_start; sc.T = T; sc.L = pl.L; sc.n_seq = pl.n_seq; sc.Hv = (int)Hv; sc.size = (int)(dk * dv);
    if ((rc = done(launch_lad_scan(sc, s))) != KDA_OK) return rc;
  }
  if (T > 0 || grads->dS0) {
    const bool shared = pl.grp > 1;
    const kda_stride_t part{Hv * T * dk, T * dk, dk};
    LadWalk a = walk_over(rdo, rv, rk), b = walk_over(rv, rdo, rq), c = walk_over(rk, rq, rdo);
    a.out = shared ? ws.dq : grads->dq; a.so = shared ? part : grads->sq; a.out_f32 = shared; a.transposed = 1;
    a.out_scale = desc->scale;
    a.entering = segments ? floats(ws.s) : S0; a.by_slot = segments;
    b.out = shared ? ws.dk : grads->dk; b.so = shared ? part : grads->sk; b.out_f32 = shared; b.transposed = 1;
    c.out = grads->dv; c.so = grads->sv;
    b.reverse = c.reverse = 1;
    b.in_scale = c.in_scale = desc->scale;
    b.entering = c.entering = segments ? floats(ws.r) : dS_final;
    b.by_slot = c.by_slot = segments;
    if (!segments) {
      a.leaving = want_end ? floats(ws.s_final) : nullptr;
      c.leaving = r_start;
    }
    const auto set_dots = [&](LadWalk& x, char* at) {
      x.dots[0] = reinterpret_cast<double*>(at);
      x.dots[1] = x.dots[0] + B * Hv * T;
    };
    if (grads->dw) {
      a.dot = q; a.sdot = desc->q; a.grp_dot = pl.grp; set_dots(a, ws.qdq);
      b.dot = k; b.sdot = desc->k; b.grp_dot = pl.grp; set_dots(b, ws.kdk);
    }
    p.walk[0] = a;
    p.walk[1] = b;
    p.walk[2] = c;
    p.n_walks = 3;
    const bool exact = (per_head && grads->dw) || a.leaving || (c.leaving && grads->dS0);
    if ((rc = done(launch_lad_bwd(p, desc->dtype, (int)dv, (int)dk, exact, s))) != KDA_OK) return rc;
    if (shared && T > 0) {
      LadSum sm{};
      sm.seq_start = seq_start; sm.B = B; sm.T = T; sm.n_seq = pl.n_seq; sm.Hk = (int)Hk; sm.grp = pl.grp; sm.D = (int)dk; sm.dtype = desc->dtype;
      sm.part[0] = floats(ws.dq); sm.out[0] = grads->dq; sm.so[0] = grads->sq;
      sm.part[1] = floats(ws.dk); sm.out[1] = grads->dk; sm.so[1] = grads->sk;
      if ((rc = done(launch_lad_sum(sm, s))) != KDA_OK) return rc;
    }
  }
  if (!grads->dw || (T == 0 && !per_head)) return KDA_OK;
  LadDecayGrad g{};
  for (int i = 0; i < 2; ++i) {
    g.qdq[i] = reinterpret_cast<const double*>(ws.qdq) + i * B * Hv * T;
    g.kdk[i] = reinterpret_cast<const double*>(ws.kdk) + i * B * Hv * T;
  }
  g.s = floats(ws.s); g.r = floats(ws.r);
  g.S0 = S0; g.S_final = floats(ws.s_final); g.dSf = dS_final; g.dS0 = r_start; g.w = w; g.sw = desc->w; g.dw = grads->dw; g.sdw = grads->sw;
  g.partial = reinterpret_cast<double*>(ws.partial); g.seq_start = seq_start;
  g.T = T; g.L = pl.L; g.n_seq = pl.n_seq; g.slots = pl.slots; g.Hv = (int)Hv; g.size = (int)(dk * dv);
  g.w_per_head = per_head; g.gate = desc->gate; g.dtype = desc->dtype; g.g_min = desc->g_min;
  return done(launch_lad_decay_grad(g, s));
}

int kda_lad_decode(const void* q, const void* k, const void* v, const void* w, float* S, int64_t n_slots, const int32_t* slots,
                   const kda_lad_t* desc, void* o, const kda_stride_t* o_stride, void* stream) {
  int rc = check_lad(desc, false);
  if (rc != KDA_OK) return rc;
  const int64_t B = desc->B, Hk = desc->Hk, Hv = desc->Hv, T = desc->T, dk = desc->dk, dv = desc->dv, e = elem(desc->dtype);
  if (n_slots < 0 || n_slots > 0x7fffffffll || (!slots && n_slots < B)) return KDA_ERR_SHAPE;
  if ((double)n_slots * Hv * dk * dv * 4 > (double)kMaxExtent) return KDA_ERR_SHAPE;
  if ((rc = check_inputs(desc, q, k, v, w)) != KDA_OK) return rc;
  if ((!S && n_slots > 0) || (T > 0 && (!o || !o_stride))) return KDA_ERR_NULL;
  const kda_stride_t so = o_stride ? *o_stride : kda_stride_t{};
  if ((rc = check_out(o, so, B, Hv, T, dv, e, 16)) != KDA_OK) return rc;
  if (!aligned(S, 16) || !aligned(slots, 4)) return KDA_ERR_ARG;
  if ((rc = check_apart({view(q, desc->q, B, Hk, T, dk, e), view(k, desc->k, B, Hk, T, dk, e), view(v, desc->v, B, Hv, T, dv, e),
                         w_span(desc, w), dense(slots, slots ? B * 4.0 : 0)},
                        {view(o, so, B, Hv, T, dv, e), dense(S, (double)n_slots * Hv * dk * dv * 4)})) != KDA_OK)
    return rc;
  if (T == 0) return KDA_OK;
  LadStepParams p{};
  p.q = q; p.k = k; p.v = v; p.w = w; p.slots = slots; p.S = S; p.o = o;
  p.sq = desc->q; p.sk = desc->k; p.sv = desc->v; p.sw = desc->w; p.so = so;
  p.B = B; p.T = T; p.n_slots = n_slots; p.Hk = (int)Hk; p.Hv = (int)Hv; p.dk = (int)dk; p.dv = (int)dv;
  p.dtype = desc->dtype; p.gate = desc->gate; p.w_per_head = desc->w_per_head; p.g_min = desc->g_min; p.scale = desc->scale;
  return done(launch_lad_step(p, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
