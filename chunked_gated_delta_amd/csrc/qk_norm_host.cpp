// Host side of the norms of queries and keys with the rotation by position: argument validation (before any HIP
// call) and launches.
#include <cmath>

#include "host_checks.h"
#include "lad_internal.h"

namespace {

using namespace kda;

int check_desc(const kda_qk_norm_t* d) {
  if (!d) return KDA_ERR_NULL;
  if (d->B < 0 || d->Hq < 0 || d->Hk < 0 || d->T < 0 || d->D < 2 || d->R < 0) return KDA_ERR_SHAPE;
  if (d->D % 2 != 0 || d->R % 2 != 0 || d->R > d->D) return KDA_ERR_SHAPE;
  if (d->D > KDA_QK_NORM_MAX_D) return KDA_ERR_UNSUPPORTED;
  if (d->Hq > 65535 || d->Hk > 65535 || (double)d->B * (double)d->T >= 2147483648.0) return KDA_ERR_SHAPE;
  // A grid holds fewer than 2^24 workgroups of 256 threads: where there are many, one takes all heads of queries or of keys
  // of its tokens, 256 / NT of them with NT lanes a row.
  const int64_t turning = (d->interleaved ? d->D : d->R) / 2, lanes = (turning + 7) / 8 + (d->D / 2 - turning + 7) / 8;
  const double tokens = lanes <= 4 ? 64 : lanes <= 8 ? 32 : lanes <= 16 ? 16 : lanes <= 32 ? 8 : 4;
  if ((double)d->B * (double)d->T / tokens >= (double)(1 << 22)) return KDA_ERR_SHAPE;
  if (d->dtype != KDA_DTYPE_F32 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
  if (d->wdtype != KDA_DTYPE_F32 && d->wdtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
  for (int32_t x : {d->norm, d->interleaved, d->wide_positions})
    if (x != 0 && x != 1) return KDA_ERR_ARG;
  if (!std::isfinite(d->q_scale) || !std::isfinite(d->k_scale) || !(d->eps >= 0.f) || !std::isfinite(d->eps)) return KDA_ERR_ARG;
  return KDA_OK;
}

// positions and frequencies; their spans
int check_angles(const kda_qk_norm_t* d, const void* positions, const float* inv_freq, Span* pos, Span* freq) {
  *pos = *freq = Span{};
  if (d->R == 0) return KDA_OK;
  if (!positions || !inv_freq) return KDA_ERR_NULL;
  const int64_t e = d->wide_positions ? 8 : 4;
  const int rc = check_strides(positions, kda_stride_t{d->pos_b, 0, d->pos_t}, d->B, 1, d->T, 1, e, e, kMaxStride);
  if (rc != KDA_OK) return rc;
  if (!aligned(inv_freq, 4)) return KDA_ERR_ARG;
  *pos = view(positions, kda_stride_t{d->pos_b, 0, d->pos_t}, d->B, 1, d->T, 1, e);
  *freq = dense(inv_freq, d->R * 2.0);
  return KDA_OK;
}

QkNormParams params(const kda_qk_norm_t* d, const void* q, const void* k, const void* qw, const void* kw, const void* positions,
                    const float* inv_freq) {
  QkNormParams p{};
  p.x[0] = q; p.x[1] = k; p.weight[0] = qw; p.weight[1] = kw;
  p.sx[0] = d->q; p.sx[1] = d->k;
  p.positions = positions; p.inv_freq = inv_freq; p.pos_b = d->pos_b; p.pos_t = d->pos_t;
  p.B = d->B; p.T = d->T; p.H[0] = (int)d->Hq; p.H[1] = (int)d->Hk; p.D = (int)d->D; p.R = (int)d->R;
  p.dtype = d->dtype; p.wdtype = d->wdtype; p.norm = d->norm; p.interleaved = d->interleaved; p.wide = d->wide_positions;
  p.scale[0] = d->q_scale; p.scale[1] = d->k_scale; p.eps = d->eps;
  return p;
}

}  // namespace

extern "C" {

size_t kda_qk_norm_bwd_workspace_bytes(const kda_qk_norm_t* desc) {
  if (check_desc(desc) != KDA_OK) return (size_t)-1;
  QkNormParams p{};
  p.D = (int)desc->D;
  return qk_norm_bwd_workspace_bytes(p);
}

int kda_qk_norm_fwd(const void* q, const void* k, const void* q_weight, const void* k_weight, const void* positions,
                    const float* inv_freq, const kda_qk_norm_t* d, void* q_out, const kda_stride_t* q_out_stride, void* k_out,
                    const kda_stride_t* k_out_stride, void* stream) {
  int rc = check_desc(d);
  if (rc != KDA_OK) return rc;
  const int64_t B = d->B, T = d->T, D = d->D, e = elem(d->dtype), we = elem(d->wdtype);
  const int64_t H[2] = {d->Hq, d->Hk};
  if (B * T * (H[0] + H[1]) == 0) return KDA_OK;
  const void* x[2] = {q, k};
  const void* w[2] = {q_weight, k_weight};
  void* y[2] = {q_out, k_out};
  const kda_stride_t sx[2] = {d->q, d->k}, *sy[2] = {q_out_stride, k_out_stride};
  Span in[6], out[2];
  for (int i = 0; i < 2; ++i) {
    if (H[i] == 0) continue;
    if (!x[i] || !y[i] || !sy[i]) return KDA_ERR_NULL;
    if ((rc = check_strides(x[i], sx[i], B, H[i], T, D, e, e, kMaxStride)) != KDA_OK) return rc;
    if ((rc = check_out(y[i], *sy[i], B, H[i], T, D, e, e, kMaxStride)) != KDA_OK) return rc;
    if (!aligned(w[i], (unsigned)we)) return KDA_ERR_ARG;
    in[2 * i] = view(x[i], sx[i], B, H[i], T, D, e);
    in[2 * i + 1] = dense(w[i], (double)D * we);
    out[i] = view(y[i], *sy[i], B, H[i], T, D, e);
  }
  if ((rc = check_angles(d, positions, inv_freq, &in[4], &in[5])) != KDA_OK) return rc;
  if ((rc = check_apart({in[0], in[1], in[2], in[3], in[4], in[5]}, {out[0], out[1]})) != KDA_OK) return rc;
  QkNormParams p = params(d, q, k, q_weight, k_weight, positions, inv_freq);
  for (int i = 0; i < 2; ++i) {
    if (H[i] == 0) p.x[i] = p.weight[i] = nullptr;
    else {
      p.y[i] = y[i];
      p.sy[i] = *sy[i];
    }
  }
  return done(launch_qk_norm_fwd(p, reinterpret_cast<hipStream_t>(stream)));
}

int kda_qk_norm_bwd(const void* q, const void* k, const void* q_weight, const void* k_weight, const void* positions,
                    const float* inv_freq, const kda_qk_norm_t* d, const void* dq_out, const kda_stride_t* dq_out_stride,
                    const void* dk_out, const kda_stride_t* dk_out_stride, const kda_qk_norm_grads_t* g, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int rc = check_desc(d);
  if (rc != KDA_OK) return rc;
  if (!g) return KDA_ERR_NULL;
  const int64_t B = d->B, T = d->T, D = d->D, e = elem(d->dtype), we = elem(d->wdtype);
  const int64_t H[2] = {d->Hq, d->Hk};
  const void *x[2] = {q, k}, *w[2] = {q_weight, k_weight}, *dy[2] = {dq_out, dk_out};
  void *dx[2] = {g->dq, g->dk}, *dw[2] = {g->dq_weight, g->dk_weight};
  const kda_stride_t sx[2] = {d->q, d->k}, sdx[2] = {g->sq, g->sk}, *sdy[2] = {dq_out_stride, dk_out_stride};
  const bool rows = B * T > 0;
  Span in[8], out[4];
  for (int i = 0; i < 2; ++i) {
    if (!w[i]) dw[i] = nullptr;
    else if (!dw[i]) return KDA_ERR_NULL;
    if (!aligned(w[i], (unsigned)we) || !aligned(dw[i], (unsigned)we)) return KDA_ERR_ARG;
    in[3 * i] = dense(w[i], (double)D * we);
    out[2 * i] = dense(dw[i], (double)D * we);
    if (!rows || H[i] == 0) continue;
    if (!x[i] || !dy[i] || !sdy[i] || !dx[i]) return KDA_ERR_NULL;
    if ((rc = check_strides(x[i], sx[i], B, H[i], T, D, e, e, kMaxStride)) != KDA_OK) return rc;
    if ((rc = check_strides(dy[i], *sdy[i], B, H[i], T, D, e, e, kMaxStride)) != KDA_OK) return rc;
    if ((rc = check_out(dx[i], sdx[i], B, H[i], T, D, e, e, kMaxStride)) != KDA_OK) return rc;
    in[3 * i + 1] = view(x[i], sx[i], B, H[i], T, D, e);
    in[3 * i + 2] = view(dy[i], *sdy[i], B, H[i], T, D, e);
    out[2 * i + 1] = view(dx[i], sdx[i], B, H[i], T, D, e);
  }
  if (rows && (rc = check_angles(d, positions, inv_freq, &in[6], &in[7])) != KDA_OK) return rc;
  QkNormParams p = params(d, q, k, q_weight, k_weight, positions, inv_freq);
  const bool sums = dw[0] || dw[1];
  const size_t need = sums ? qk_norm_bwd_workspace_bytes(p) : 0;
  if (sums && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return KDA_ERR_ARG;
  if ((rc = check_apart({in[0], in[1], in[2], in[3], in[4], in[5], in[6], in[7]},
                        {out[0], out[1], out[2], out[3], dense(workspace, (double)need)})) != KDA_OK)
    return rc;
  for (int i = 0; i < 2; ++i) {
    p.dweight[i] = dw[i];
    if (!rows || H[i] == 0) {
      p.x[i] = nullptr;
      p.H[i] = 0;
      continue;
    }
    p.dy[i] = dy[i];
    p.sdy[i] = *sdy[i];
    p.dx[i] = dx[i];
    p.sdx[i] = sdx[i];
  }
  p.partial = static_cast<float*>(workspace);
  return done(launch_qk_norm_bwd(p, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
