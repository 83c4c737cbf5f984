// Host side of the head-gated delta rule and of the norms around a block: argument validation (before
// any HIP call), workspace layout, launches.
#include <cmath>

#include "host_checks.h"

namespace {

using namespace kda;

// sizes, types and the gate.  Launch limits: a grid holds fewer than 2^24 workgroups of 256 threads
int check_gdr(const kda_gdr_t* d, bool packed) {
  if (!d) return KDA_ERR_NULL;
  if (d->B < 1 || d->Hk < 1 || d->Hv < 1 || d->T < 0 || d->dk < 1 || d->dv < 1) return KDA_ERR_SHAPE;
  if (d->Hk > 65535 || d->Hv > 65535 || d->Hv % d->Hk != 0) return KDA_ERR_SHAPE;
  if (d->T > 0x7fffffffll || d->B > 0x7fffffffll) return KDA_ERR_SHAPE;
  if (packed ? (d->B != 1 || d->n_seq < 1 || d->n_seq > 0x7fffffffll) : d->n_seq != 0) return KDA_ERR_SHAPE;
  if (!head_dim(d->dk) || !head_dim(d->dv)) return KDA_ERR_UNSUPPORTED;
  if (d->dtype != KDA_DTYPE_F32 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
  if (d->gate != KDA_GATE_BOUNDED && d->gate != KDA_GATE_SOFTPLUS && d->gate != KDA_GATE_LOG) return KDA_ERR_UNSUPPORTED;
  if (d->gate == KDA_GATE_BOUNDED && !(d->g_min <= 0.f && std::isfinite(d->g_min))) return KDA_ERR_ARG;
  if (!std::isfinite(d->scale)) return KDA_ERR_ARG;
  const int64_t n_seq = packed ? d->n_seq : d->B;
  const double slots = (double)kda::gdr_slots(d->B, d->T, n_seq, packed);
  if (slots >= (double)(1 << 24) || (double)n_seq * d->Hv * (d->dv / 16) >= (double)(1 << 23)) return KDA_ERR_SHAPE;
  if (slots * d->Hv * (double)(d->dk * d->dv) * 4.0 > (double)kMaxExtent) return KDA_ERR_SHAPE;
  return KDA_OK;
}

// and the launches of the chunked kernels, of 512 threads: a grid holds fewer than 2^23 of them
int check_chunked(const kda_gdr_t* d, bool packed, bool bwd) {
  const int rc = check_gdr(d, packed);
  if (rc != KDA_OK) return rc;
  const int64_t n_seq = packed ? d->n_seq : d->B, most = (int64_t)1 << 23;
  if (kda::gdr_blocks(n_seq * d->Hv, (int)(d->dv / 16)) >= most) return KDA_ERR_SHAPE;
  return bwd && kda::gdr_slots(d->B, d->T, n_seq, packed) >= most ? KDA_ERR_SHAPE : KDA_OK;
}

int check_gdr_inputs(const kda_gdr_t* d, const void* q, const void* k, const void* v, const void* w, const void* beta) {
  const int64_t B = d->B, T = d->T, e = elem(d->dtype);
  if (T > 0 && (!q || !k || !v || !w || !beta)) return KDA_ERR_NULL;
  int rc;
  if ((rc = check_strides(q, d->q, B, d->Hk, T, d->dk, e, 16)) != KDA_OK) return rc;
  if ((rc = check_strides(k, d->k, B, d->Hk, T, d->dk, e, 16)) != KDA_OK) return rc;
  if ((rc = check_strides(v, d->v, B, d->Hv, T, d->dv, e, 16)) != KDA_OK) return rc;
  if ((rc = check_strides(w, d->w, B, d->Hv, T, 1, e, e)) != KDA_OK) return rc;
  return check_strides(beta, d->beta, B, d->Hv, T, 1, e, e);
}

kda::GdrParams gdr_params(const kda_gdr_t* d, const void* q, const void* k, const void* v, const void* w, const void* beta,
                          const float* S0, const int32_t* seq_start) {
  kda::GdrParams p{};
  p.q = q; p.k = k; p.v = v; p.w = w; p.beta = beta; p.S0 = S0; p.seq_start = seq_start;
  p.sq = d->q; p.sk = d->k; p.sv = d->v; p.sw = d->w; p.sb = d->beta;
  p.B = d->B; p.T = d->T; p.n_seq = seq_start ? d->n_seq : d->B;
  p.Hk = (int)d->Hk; p.Hv = (int)d->Hv; p.dk = (int)d->dk; p.dv = (int)d->dv;
  p.dtype = d->dtype; p.gate = d->gate; p.g_min = d->g_min; p.scale = d->scale;
  return p;
}

}  // namespace

namespace kda {

int64_t gdr_slots(int64_t B, int64_t T, int64_t n_seq, bool packed) {
  return packed ? T / kGdrChunk + n_seq : B * ((T + kGdrChunk - 1) / kGdrChunk);
}

size_t gdr_layout(GdrParams& p, void* base, bool bwd) {
  const size_t slots = (size_t)gdr_slots(p.B, p.T, p.n_seq, p.seq_start != nullptr);
  const size_t e = p.dtype == KDA_DTYPE_BF16 ? 2 : 4, op = (e == 2 ? 3 : 2) * kPlane;
  const size_t vh = slots * p.Hv;
  size_t off = 0;
  auto take = [&](char*& at, size_t bytes) {
    at = base ? static_cast<char*>(base) + off : nullptr;
    off += (bytes + 255) / 256 * 256;
  };
  take(p.ws_gate, vh * kGateFloats * 4);
  take(p.ws_ti, vh * kTriFrags * op);
  take(p.ws_p, vh * kTriFrags * (bwd ? op : 2 * kPlane));
  if (bwd) {
    take(p.ws_tt, vh * kTriFrags * op);
    take(p.ws_s, vh * p.dk * p.dv * 4);    // fp32, or two planes of bf16
    take(p.ws_ds, vh * p.dk * p.dv * 4);
    take(p.ws_f, vh * kGdrChunk * p.dv * 4);
    take(p.ws_e, e == 2 ? vh * kGdrChunk * p.dv * 2 : 0);   // the second plane of dv
    take(p.ws_db, vh * (p.dv / 16) * kGdrChunk * 4);
  }
  return off;
}

}  // namespace kda

extern "C" {

size_t kda_gdr_workspace_bytes(const kda_gdr_t* desc, int backward) {
  if (!desc || check_chunked(desc, desc->n_seq != 0, backward != 0) != KDA_OK) return (size_t)-1;
  if (desc->T == 0) return 0;
  static const int32_t packed = 0;
  kda::GdrParams p = gdr_params(desc, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, desc->n_seq ? &packed : nullptr);
  return kda::gdr_layout(p, nullptr, backward != 0);
}

int kda_gdr_chunk_fwd(const void* q, const void* k, const void* v, const void* w, const void* beta, const float* S0,
                      const int32_t* seq_start, const kda_gdr_t* desc, void* o, const kda_stride_t* o_stride, float* S_final,
                      void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_chunked(desc, seq_start != nullptr, false);
  if (rc != KDA_OK) return rc;
  const int64_t B = desc->B, Hk = desc->Hk, Hv = desc->Hv, T = desc->T, dk = desc->dk, dv = desc->dv, e = elem(desc->dtype);
  if ((rc = check_gdr_inputs(desc, q, k, v, w, beta)) != KDA_OK) return rc;
  if (T > 0 && (!o || !o_stride)) return KDA_ERR_NULL;
  const kda_stride_t so = o_stride ? *o_stride : kda_stride_t{};
  if ((rc = check_out(o, so, B, Hv, T, dv, e, 16)) != KDA_OK) return rc;
  if (!aligned(S0, 16) || !aligned(S_final, 16) || !aligned(workspace, 16) || !aligned(seq_start, 4)) return KDA_ERR_ARG;
  kda::GdrParams p = gdr_params(desc, q, k, v, w, beta, S0, seq_start);
  const size_t need = T > 0 ? kda::gdr_layout(p, workspace, false) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_ARG;
  const double states = (double)p.n_seq * Hv * dk * dv * 4;
  const Span s0 = dense(S0, states), sf = dense(S_final, states), out = view(o, so, B, Hv, T, dv, e), ws = dense(workspace, (double)need);
  const Span start = dense(seq_start, seq_start ? (desc->n_seq + 1) * 4.0 : 0);
  if ((rc = check_apart({view(q, desc->q, B, Hk, T, dk, e), view(k, desc->k, B, Hk, T, dk, e), view(v, desc->v, B, Hv, T, dv, e),
                         view(w, desc->w, B, Hv, T, 1, e), view(beta, desc->beta, B, Hv, T, 1, e), start},
                        {out, sf, ws})) != KDA_OK)
    return rc;
  if (meet(s0, out) || meet(s0, ws) || (S0 != S_final && meet(s0, sf))) return KDA_ERR_ARG;   // S_final may be S0
  p.o = o; p.so = so; p.S_final = S_final;
  return done(kda::launch_gdr_fwd(p, reinterpret_cast<hipStream_t>(stream)));
}

int kda_gdr_chunk_bwd(const void* q, const void* k, const void* v, const void* w, const void* beta, const float* S0,
                      const int32_t* seq_start, const kda_gdr_t* desc, const void* dO, const kda_stride_t* dO_stride,
                      const float* dS_final, const kda_gdr_grads_t* grads, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int rc = check_chunked(desc, seq_start != nullptr, true);
  if (rc != KDA_OK) return rc;
  if (!grads) return KDA_ERR_NULL;
  const int64_t B = desc->B, Hk = desc->Hk, Hv = desc->Hv, T = desc->T, dk = desc->dk, dv = desc->dv, e = elem(desc->dtype);
  if ((rc = check_gdr_inputs(desc, q, k, v, w, beta)) != KDA_OK) return rc;
  if (T > 0 && (!dO || !dO_stride || !grads->dq || !grads->dk || !grads->dv || !grads->dw || !grads->dbeta)) return KDA_ERR_NULL;
  const kda_stride_t sdo = dO_stride ? *dO_stride : kda_stride_t{};
  if ((rc = check_strides(dO, sdo, B, Hv, T, dv, e, 16)) != KDA_OK) return rc;
  if ((rc = check_out(grads->dq, grads->sq, B, Hk, T, dk, e, 16)) != KDA_OK) return rc;
  if ((rc = check_out(grads->dk, grads->sk, B, Hk, T, dk, e, 16)) != KDA_OK) return rc;
  if ((rc = check_out(grads->dv, grads->sv, B, Hv, T, dv, e, 16)) != KDA_OK) return rc;
  if ((rc = check_out(grads->dw, grads->sw, B, Hv, T, 1, e, e)) != KDA_OK) return rc;
  if ((rc = check_out(grads->dbeta, grads->sbeta, B, Hv, T, 1, e, e)) != KDA_OK) return rc;
  if (!aligned(S0, 16) || !aligned(dS_final, 16) || !aligned(grads->dS0, 16) || !aligned(workspace, 16) || !aligned(seq_start, 4))
    return KDA_ERR_ARG;
  kda::GdrParams p = gdr_params(desc, q, k, v, w, beta, S0, seq_start);
  const size_t need = T > 0 ? kda::gdr_layout(p, workspace, true) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_ARG;
  const double states = (double)p.n_seq * Hv * dk * dv * 4;
  if ((rc = check_apart({view(q, desc->q, B, Hk, T, dk, e), view(k, desc->k, B, Hk, T, dk, e), view(v, desc->v, B, Hv, T, dv, e),
                         view(w, desc->w, B, Hv, T, 1, e), view(beta, desc->beta, B, Hv, T, 1, e),
                         dense(seq_start, seq_start ? (desc->n_seq + 1) * 4.0 : 0), view(dO, sdo, B, Hv, T, dv, e), dense(S0, states),
                         dense(dS_final, states)},
                        {view(grads->dq, grads->sq, B, Hk, T, dk, e), view(grads->dk, grads->sk, B, Hk, T, dk, e),
                         view(grads->dv, grads->sv, B, Hv, T, dv, e), view(grads->dw, grads->sw, B, Hv, T, 1, e),
                         view(grads->dbeta, grads->sbeta, B, Hv, T, 1, e), dense(grads->dS0, states),
                         dense(workspace, (double)need)})) != KDA_OK)
    return rc;
  p.dO = dO; p.sdo = sdo; p.dSf = dS_final;
  p.dq = grads->dq; p.dk_ = grads->dk; p.dv_ = grads->dv; p.dw = grads->dw; p.dbeta = grads->dbeta; p.dS0 = grads->dS0;
  p.sdq = grads->sq; p.sdk = grads->sk; p.sdv = grads->sv; p.sdw = grads->sw; p.sdb = grads->sbeta;
  return done(kda::launch_gdr_bwd(p, reinterpret_cast<hipStream_t>(stream)));
}

int kda_gdr_decode(const void* q, const void* k, const void* v, const void* w, const void* beta, float* S, int64_t n_slots,
                   const int32_t* slots, const kda_gdr_t* desc, void* o, const kda_stride_t* o_stride, void* stream) {
  int rc = check_gdr(desc, false);
  if (rc != KDA_OK) return rc;
  const int64_t B = desc->B, Hk = desc->Hk, Hv = desc->Hv, T = desc->T, dk = desc->dk, dv = desc->dv, e = elem(desc->dtype);
  if (n_slots < 0 || n_slots > 0x7fffffffll || (!slots && n_slots < B)) return KDA_ERR_SHAPE;
  if ((double)n_slots * Hv * dk * dv * 4 > (double)kMaxExtent) return KDA_ERR_SHAPE;
  if ((rc = check_gdr_inputs(desc, q, k, v, w, beta)) != KDA_OK) return rc;
  if ((!S && n_slots > 0) || (T > 0 && (!o || !o_stride))) return KDA_ERR_NULL;
  const kda_stride_t so = o_stride ? *o_stride : kda_stride_t{};
  if ((rc = check_out(o, so, B, Hv, T, dv, e, 16)) != KDA_OK) return rc;
  if (!aligned(S, 16) || !aligned(slots, 4)) return KDA_ERR_ARG;
  if ((rc = check_apart({view(q, desc->q, B, Hk, T, dk, e), view(k, desc->k, B, Hk, T, dk, e), view(v, desc->v, B, Hv, T, dv, e),
                         view(w, desc->w, B, Hv, T, 1, e), view(beta, desc->beta, B, Hv, T, 1, e), dense(slots, slots ? B * 4.0 : 0)},
                        {view(o, so, B, Hv, T, dv, e), dense(S, (double)n_slots * Hv * dk * dv * 4)})) != KDA_OK)
    return rc;
  if (T == 0) return KDA_OK;
  kda::GdrStepParams p{};
  p.q = q; p.k = k; p.v = v; p.w = w; p.beta = beta; p.slots = slots; p.S = S; p.o = o;
  p.sq = desc->q; p.sk = desc->k; p.sv = desc->v; p.sw = desc->w; p.sb = desc->beta; p.so = so;
  p.B = B; p.T = T; p.n_slots = n_slots; p.Hk = (int)Hk; p.Hv = (int)Hv; p.dk = (int)dk; p.dv = (int)dv;
  p.dtype = desc->dtype; p.gate = desc->gate; p.g_min = desc->g_min; p.scale = desc->scale;
  return done(kda::launch_gdr_step(p, reinterpret_cast<hipStream_t>(stream)));
}

static int check_norm(const kda_norm_t* d) {
  if (!d) return KDA_ERR_NULL;
  if (d->B < 0 || d->H < 0 || d->T < 0 || d->D < 1) return KDA_ERR_SHAPE;
  if (d->D > KDA_NORM_MAX_D) return KDA_ERR_UNSUPPORTED;
  // one workgroup a row at most, and a grid of fewer than 2^23 of 512 threads
  if ((double)d->B * d->H * d->T >= (double)(1 << 23) * (d->D <= 128 ? 16 : d->D <= 1024 ? 4 : 1)) return KDA_ERR_SHAPE;
  if (d->dtype != KDA_DTYPE_F32 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
  if (d->wdtype != KDA_DTYPE_F32 && d->wdtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
  if (d->act != KDA_ACT_SIGMOID && d->act != KDA_ACT_SILU) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(d->alpha) || !(d->eps >= 0.f) || !std::isfinite(d->eps)) return KDA_ERR_ARG;
  return KDA_OK;
}

size_t kda_norm_bwd_workspace_bytes(const kda_norm_t* desc) {
  if (check_norm(desc) != KDA_OK) return (size_t)-1;
  kda::NormParams p{};
  p.D = desc->D;
  return kda::norm_bwd_workspace_bytes(p);
}

int kda_norm_fwd(const void* x, const void* weight, const void* z, const void* residual, const void* next_weight,
                 const kda_norm_t* d, void* s, const kda_stride_t* s_stride, void* y, const kda_stride_t* y_stride,
                 void* stream) {
  int rc = check_norm(d);
  if (rc != KDA_OK) return rc;
  if (!weight && !next_weight) return KDA_ERR_ARG;   // no norm asked for
  const int64_t B = d->B, H = d->H, T = d->T, D = d->D, e = elem(d->dtype), we = elem(d->wdtype);
  if (B * H * T == 0) return KDA_OK;
  if (!x || !s || !s_stride || (next_weight && (!y || !y_stride))) return KDA_ERR_NULL;
  if (!next_weight) y = nullptr;
  const kda_stride_t sy = y ? *y_stride : kda_stride_t{};
  if ((rc = check_strides(x, d->x, B, H, T, D, e, e, kMaxStride)) != KDA_OK) return rc;
  if ((rc = check_strides(z, d->z, B, H, T, D, e, e, kMaxStride)) != KDA_OK) return rc;
  if ((rc = check_strides(residual, d->residual, B, H, T, D, e, e, kMaxStride)) != KDA_OK) return rc;
  if ((rc = check_out(s, *s_stride, B, H, T, D, e, e, kMaxStride)) != KDA_OK) return rc;
  if ((rc = check_out(y, sy, B, H, T, D, e, e, kMaxStride)) != KDA_OK) return rc;
  if (!aligned(weight, (unsigned)we) || !aligned(next_weight, (unsigned)we)) return KDA_ERR_ARG;
  if ((rc = check_apart({view(x, d->x, B, H, T, D, e), view(z, d->z, B, H, T, D, e), view(residual, d->residual, B, H, T, D, e),
                         dense(weight, (double)D * we), dense(next_weight, (double)D * we)},
                        {view(s, *s_stride, B, H, T, D, e), view(y, sy, B, H, T, D, e)})) != KDA_OK)
    return rc;
  kda::NormParams p{};
  p.x = x; p.z = z; p.res = residual; p.weight = weight; p.weight2 = next_weight; p.s = s; p.y = y;
  p.sx = d->x; p.sz = d->z; p.sr = d->residual; p.ss = *s_stride; p.sy = sy;
  p.B = B; p.H = H; p.T = T; p.D = D; p.dtype = d->dtype; p.wdtype = d->wdtype; p.act = d->act; p.alpha = d->alpha; p.eps = d->eps;
  return done(kda::launch_norm_fwd(p, reinterpret_cast<hipStream_t>(stream)));
}

int kda_norm_bwd(const void* x, const void* weight, const void* z, const void* residual, const void* next_weight,
                 const kda_norm_t* d, const void* ds, const kda_stride_t* ds_stride, const void* dy, const kda_stride_t* dy_stride,
                 const kda_norm_grads_t* g, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_norm(d);
  if (rc != KDA_OK) return rc;
  if (!weight && !next_weight) return KDA_ERR_ARG;
  if (!g) return KDA_ERR_NULL;
  const int64_t B = d->B, H = d->H, T = d->T, D = d->D, e = elem(d->dtype), we = elem(d->wdtype);
  const bool rows = B * H * T > 0;
  if (rows && (!x || !g->dx || (z && !g->dz) || (residual && !g->dresidual))) return KDA_ERR_NULL;
  if (rows && ((ds && !ds_stride) || (next_weight ? !dy || !dy_stride : !ds))) return KDA_ERR_NULL;
  if ((weight && !g->dweight) || (next_weight && !g->dnext_weight)) return KDA_ERR_NULL;
  const kda_stride_t none{}, sds = ds_stride ? *ds_stride : none, sdy = dy_stride ? *dy_stride : none;
  if (!next_weight) dy = nullptr;
  void *dz = z ? g->dz : nullptr, *dres = residual ? g->dresidual : nullptr;
  void *dwt = weight ? g->dweight : nullptr, *dw2 = next_weight ? g->dnext_weight : nullptr;
  const struct { const void* p; kda_stride_t s; } ins[] = {{x, d->x}, {z, d->z}, {residual, d->residual}, {ds, sds}, {dy, sdy}};
  for (const auto& t : ins)
    if ((rc = check_strides(t.p, t.s, B, H, T, D, e, e, kMaxStride)) != KDA_OK) return rc;
  const struct { const void* p; kda_stride_t s; } outs[] = {{g->dx, g->sx}, {dz, g->sz}, {dres, g->sresidual}};
  for (const auto& t : outs)
    if ((rc = check_out(t.p, t.s, B, H, T, D, e, e, kMaxStride)) != KDA_OK) return rc;
  for (const void* q : {weight, next_weight, (const void*)dwt, (const void*)dw2})
    if (!aligned(q, (unsigned)we)) return KDA_ERR_ARG;
  kda::NormParams p{};
  p.D = D;
  const size_t need = kda::norm_bwd_workspace_bytes(p);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return KDA_ERR_ARG;
  if ((rc = check_apart({view(x, d->x, B, H, T, D, e), view(z, d->z, B, H, T, D, e), view(residual, d->residual, B, H, T, D, e),
                         view(ds, sds, B, H, T, D, e), view(dy, sdy, B, H, T, D, e), dense(weight, (double)D * we),
                         dense(next_weight, (double)D * we)},
                        {view(g->dx, g->sx, B, H, T, D, e), view(dz, g->sz, B, H, T, D, e), view(dres, g->sresidual, B, H, T, D, e),
                         dense(dwt, (double)D * we), dense(dw2, (double)D * we), dense(workspace, (double)need)})) != KDA_OK)
    return rc;
  p.x = x; p.z = z; p.res = residual; p.weight = weight; p.weight2 = next_weight; p.ds = ds; p.dy = dy;
  p.sx = d->x; p.sz = d->z; p.sr = d->residual; p.sds = sds; p.sdy = sdy;
  p.dx = g->dx; p.dz = dz; p.dres = dres; p.dweight = dwt; p.dweight2 = dw2;
  p.sdx = g->sx; p.sdz = g->sz; p.sdr = g->sresidual;
  p.partial = static_cast<float*>(workspace);
  p.B = B; p.H = H; p.T = T; p.dtype = d->dtype; p.wdtype = d->wdtype; p.act = d->act; p.alpha = d->alpha; p.eps = d->eps;
  return done(kda::launch_norm_bwd(p, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace kda {

hipError_t launch_gdr_fwd(const GdrParams& p, hipStream_t s) {
  hipError_t e = launch_gdr_prep(p, s, false);
  return e != hipSuccess ? e : launch_gdr_scan(p, s, false);
}

hipError_t launch_gdr_bwd(const GdrParams& p, hipStream_t s) {
  hipError_t e = launch_gdr_prep(p, s, true);
  if (e == hipSuccess) e = launch_gdr_scan(p, s, true);
  if (e == hipSuccess) e = launch_gdr_rscan(p, s);
  if (e == hipSuccess) e = launch_gdr_grad(p, s);
  return e;
}

}  // namespace kda
