// seq_api.hip -- the extern "C" entry points of the sequence-to-sequence
// operators (include/lstm.h): argument checks, then the launches.
#include <math.h>

#include "attend_common.hpp"
#include "internal.hpp"
#include "seq_internal.hpp"

namespace lstm {

static bool dtype_ok(int d) { return d == LSTM_F32 || d == LSTM_BF16 || d == LSTM_F16; }
static bool id_ok(int t) { return t == LSTM_I32 || t == LSTM_I64; }
// a softmax's scale: scale log2 e is a positive number
static bool scale_ok(float s) { return s > 0.f && s <= 2.3e38f; }
static bool off_size(const void* p, int64_t e) { return p && ((uintptr_t)p % (uintptr_t)e) != 0; }
static int status(hipError_t e) { return e == hipSuccess ? LSTM_OK : LSTM_ERR_LAUNCH; }
static int64_t esize_of(int dtype) { return dtype == LSTM_F32 ? 4 : 2; }

static int embed_plan(const lstm_embed_shape* s, EmbedPlan* p) {
  if (!s) return LSTM_ERR_NULL;
  if (s->N < 0 || s->V < 0 || s->D < 0 || s->ld_table < s->D || s->ld_out < s->D || s->padding < -1 ||
      s->padding >= (s->V > 0 ? s->V : 1) || !(fabsf(s->scale) <= 3.4028234e38f))
    return LSTM_ERR_DIMS;
  if (!dtype_ok(s->dtype) || !id_ok(s->id_type)) return LSTM_ERR_DTYPE;
  const int64_t lim = (int64_t)1 << 26, far = (int64_t)1 << 36;  // row strides: offsets fit 63 bits
  if (s->N >= lim || s->V >= lim || s->D > ((int64_t)1 << 20) || s->ld_table >= far || s->ld_out >= far)
    return LSTM_ERR_UNSUPPORTED;
  int cus = 0;
  const int rc = device_cus(&cus, nullptr);
  if (rc != LSTM_OK) return rc;
  make_embed_plan(*s, p);
  return LSTM_OK;
}

static int logprob_plan(const lstm_logprob_shape* s, LogprobPlan* p) {
  if (!s) return LSTM_ERR_NULL;
  if (s->N < 0 || s->V < 0 || s->ld < s->V || s->ld_grad < s->V || s->top < 0 || s->top > LSTM_MAX_TOP ||
      s->top > s->V || !scale_ok(s->scale))
    return LSTM_ERR_DIMS;
  if (!dtype_ok(s->dtype) || !id_ok(s->id_type)) return LSTM_ERR_DTYPE;
  const int64_t far = (int64_t)1 << 36;
  if (s->N >= ((int64_t)1 << 24) || s->V >= ((int64_t)1 << 30) || s->ld >= far || s->ld_grad >= far ||
      (s->V > 0 && s->N >= ((int64_t)1 << 37) / s->V))
    return LSTM_ERR_UNSUPPORTED;
  int cus = 0;
  const int rc = device_cus(&cus, nullptr);
  if (rc != LSTM_OK) return rc;
  make_logprob_plan(*s, cus, p);
  return LSTM_OK;
}

// A tensor of [T][B][H] rows of D values whose rows do not overlap.
static bool disjoint(const lstm_stride& s, int64_t T, int64_t B, int64_t H, int64_t D) {
  if (T == 0 || B == 0 || H == 0) return true;
  int64_t st[3] = {s.t, s.b, s.h}, n[3] = {T, B, H}, cover = D;
  for (int i = 0; i < 3; ++i) {
    int k = -1;
    for (int j = 0; j < 3; ++j)
      if (n[j] > 1 && (k < 0 || st[j] < st[k])) k = j;
    if (k < 0) return true;
    if (st[k] < cover) return false;
    cover += st[k] * (n[k] - 1);
    n[k] = 1;
  }
  return true;
}
static bool strides_ok(const lstm_stride& s) {
  const int64_t far = (int64_t)1 << 36;
  return s.t >= 0 && s.b >= 0 && s.h >= 0 && s.t < far && s.b < far && s.h < far;
}
// whole aligned 16-byte chunks in every row
static bool whole_rows(const void* p, const lstm_stride& s, int64_t D, int64_t e) {
  return aligned16(p) && (D * e) % 16 == 0 && (s.t * e) % 16 == 0 && (s.b * e) % 16 == 0 && (s.h * e) % 16 == 0;
}
// rows a tile of which can be loaded through one descriptor
static bool dma_rows(const void* p, const lstm_stride& s, int64_t D, int64_t e) {
  return whole_rows(p, s, D, e) && s.t >= D && s.t * e < ((int64_t)1 << 31) / 64;
}

static int attend_plan(const lstm_attend_shape* s, bool bwd, AttendPlan* p) {
  if (!s) return LSTM_ERR_NULL;
  if (s->Tq < 0 || s->Tk < 0 || s->B < 0 || s->Hq < 0 || s->Hk < 0 || s->D < 1 || (s->Hk == 0) != (s->Hq == 0) ||
      (s->Hk > 0 && s->Hq % s->Hk != 0) || !scale_ok(s->scale) || s->mask_b < 0 ||
      !strides_ok(s->q) || !strides_ok(s->k) || !strides_ok(s->v) || !strides_ok(s->o) ||
      !disjoint(s->o, s->Tq, s->B, s->Hq, s->D))
    return LSTM_ERR_DIMS;
  if (bwd && (!strides_ok(s->dout) || !strides_ok(s->dq) || !strides_ok(s->dk) || !strides_ok(s->dv) ||
              !disjoint(s->dq, s->Tq, s->B, s->Hq, s->D) || !disjoint(s->dk, s->Tk, s->B, s->Hk, s->D) ||
              !disjoint(s->dv, s->Tk, s->B, s->Hk, s->D)))
    return LSTM_ERR_DIMS;
  if (!dtype_ok(s->dtype)) return LSTM_ERR_DTYPE;
  const int64_t big = (int64_t)1 << 26, wide = (int64_t)1 << 20;
  if (s->D > 256 || s->Tq >= big || s->Tk >= big || s->B >= wide || s->Hq >= wide || s->mask_b >= ((int64_t)1 << 36))
    return LSTM_ERR_UNSUPPORTED;
  const int64_t G = s->Hk > 0 ? s->Hq / s->Hk : 1, M = s->Tq * G, groups = s->B * s->Hk + 8;
  // work-groups of any launch stay below 2^24
  if (M >= ((int64_t)1 << 30) || groups >= ((int64_t)1 << 23) || groups * ((M + 31) / 32 + 64) >= ((int64_t)1 << 24) ||
      groups * ((s->Tk + 127) / 128) >= ((int64_t)1 << 24))
    return LSTM_ERR_UNSUPPORTED;
  int cus = 0;
  const int rc = device_cus(&cus, nullptr);
  if (rc != LSTM_OK) return rc;
  make_attend_plan(*s, cus, p);
  return LSTM_OK;
}

static AttendArgs attend_args(const lstm_attend_shape& s) {
  AttendArgs a = {};
  a.qs = s.q; a.ks = s.k; a.vs = s.v; a.os = s.o; a.gs = s.dout; a.dqs = s.dq; a.dks = s.dk; a.dvs = s.dv;
  a.mask_b = s.mask_b;
  a.Tq = (int)s.Tq; a.Tk = (int)s.Tk; a.B = (int)s.B; a.Hq = (int)s.Hq; a.Hk = (int)s.Hk;
  a.G = s.Hk > 0 ? (int)(s.Hq / s.Hk) : 1;
  a.D = (int)s.D;
  a.M = (uint32_t)(s.Tq * a.G);
  if (s.Hk == 0) a.M = 0;
  a.scale = s.scale;
  return a;
}

}  // namespace lstm

using namespace lstm;

extern "C" {

int lstm_embed_query(const lstm_embed_shape* shape, size_t* workspace_bytes) {
  if (!workspace_bytes) return LSTM_ERR_NULL;
  EmbedPlan p;
  const int rc = embed_plan(shape, &p);
  if (rc != LSTM_OK) return rc;
  *workspace_bytes = p.total;
  return LSTM_OK;
}

int lstm_embed_fwd(const lstm_embed_shape* shape, const void* ids, const void* table, void* out, void* stream) {
  EmbedPlan p;
  const int rc = embed_plan(shape, &p);
  if (rc != LSTM_OK) return rc;
  const bool any = p.N > 0 && p.D > 0;
  if (any && (!ids || !out || (p.V > 0 && !table))) return LSTM_ERR_NULL;
  const int64_t e = esize_of(p.dtype);
  if (off_size(ids, p.id64 ? 8 : 4) || off_size(table, e) || off_size(out, e)) return LSTM_ERR_ALIGN;
  return status(launch_embed_fwd(p, ids, table, out, (hipStream_t)stream));
}

int lstm_embed_bwd(const lstm_embed_shape* shape, const void* ids, const void* dout, void* workspace,
                   size_t workspace_bytes, void* dtable, void* stream) {
  EmbedPlan p;
  const int rc = embed_plan(shape, &p);
  if (rc != LSTM_OK) return rc;
  const bool any = p.V > 0 && p.D > 0;
  if (any && (!dtable || (p.N > 0 && (!ids || !dout)) || (p.total > 0 && !workspace))) return LSTM_ERR_NULL;
  const int64_t e = esize_of(p.dtype);
  if (off_size(ids, p.id64 ? 8 : 4) || off_size(dout, e) || off_size(dtable, e) || ((uintptr_t)workspace & 255u))
    return LSTM_ERR_ALIGN;
  if (any && workspace_bytes < p.total) return LSTM_ERR_WORKSPACE;
  return status(launch_embed_bwd(p, ids, dout, (char*)workspace, dtable, (hipStream_t)stream));
}

int lstm_logprob_query(const lstm_logprob_shape* shape, size_t* workspace_bytes) {
  if (!workspace_bytes) return LSTM_ERR_NULL;
  LogprobPlan p;
  const int rc = logprob_plan(shape, &p);
  if (rc != LSTM_OK) return rc;
  *workspace_bytes = p.total;
  return LSTM_OK;
}

int lstm_logprob_fwd(const lstm_logprob_shape* shape, const void* logits, const void* targets, void* workspace,
                     size_t workspace_bytes, float* record, float* lse, float* logp, float* entropy, float* top_logp,
                     void* top_ids, void* stream) {
  LogprobPlan p;
  const int rc = logprob_plan(shape, &p);
  if (rc != LSTM_OK) return rc;
  if (p.N > 0 && (!record || (p.V > 0 && !logits) || (logp && !targets) || (p.top > 0 && (!top_logp || !top_ids)) ||
                  (p.total > 0 && !workspace)))
    return LSTM_ERR_NULL;
  const int64_t ids = p.id64 ? 8 : 4;
  if (off_size(logits, esize_of(p.dtype)) || off_size(targets, ids) || off_size(record, 4) ||
      off_size(lse, 4) || off_size(logp, 4) || off_size(entropy, 4) || off_size(top_logp, 4) || off_size(top_ids, ids) || ((uintptr_t)workspace & 255u))
    return LSTM_ERR_ALIGN;
  if (workspace_bytes < p.total) return LSTM_ERR_WORKSPACE;
  return status(launch_logprob_fwd(p, logits, targets, (char*)workspace, record, lse, logp, entropy, top_logp, top_ids,
                                   (hipStream_t)stream));
}

int lstm_logprob_bwd(const lstm_logprob_shape* shape, const void* logits, const void* targets, const float* record,
                     const float* entropy, const void* top_ids, const float* dlogp, const float* dentropy,
                     const float* dtop, void* dlogits, void* stream) {
  LogprobPlan p;
  const int rc = logprob_plan(shape, &p);
  if (rc != LSTM_OK) return rc;
  if (p.N > 0 && p.V > 0 &&
      (!logits || !dlogits || !record || (dlogp && !targets) || (dentropy && !entropy) || (dtop && p.top > 0 && !top_ids)))
    return LSTM_ERR_NULL;
  const int64_t ids = p.id64 ? 8 : 4, e = esize_of(p.dtype);
  if (off_size(logits, e) || off_size(dlogits, e) || off_size(targets, ids) || off_size(record, 4) ||
      off_size(entropy, 4) || off_size(top_ids, ids) || off_size(dlogp, 4) || off_size(dentropy, 4) ||
      off_size(dtop, 4))
    return LSTM_ERR_ALIGN;
  if (dlogits == logits && p.ld != p.ldg) return LSTM_ERR_DIMS;
  return status(launch_logprob_bwd(p, logits, targets, record, entropy, top_ids, dlogp, dentropy, dtop, dlogits,
                                   (hipStream_t)stream));
}

int lstm_attend_query(const lstm_attend_shape* shape, size_t* fwd_bytes, size_t* bwd_bytes) {
  if (!fwd_bytes || !bwd_bytes) return LSTM_ERR_NULL;
  AttendPlan p;
  const int rc = attend_plan(shape, false, &p);
  if (rc != LSTM_OK) return rc;
  *fwd_bytes = p.total_fwd;
  *bwd_bytes = p.total_bwd;
  return LSTM_OK;
}

int lstm_attend_fwd(const lstm_attend_shape* shape, const void* q, const void* k, const void* v, const void* k_length,
                    const void* key_mask, void* workspace, size_t workspace_bytes, void* o, float* lse, void* stream) {
  AttendPlan p;
  const int rc = attend_plan(shape, false, &p);
  if (rc != LSTM_OK) return rc;
  AttendArgs a = attend_args(*shape);
  const bool any = a.M > 0 && a.B > 0;
  if (any && (!q || !o || !lse || (a.Tk > 0 && (!k || !v)) || (p.total_fwd > 0 && !workspace))) return LSTM_ERR_NULL;
  const int64_t e = esize_of(p.dtype);
  if (off_size(q, e) || off_size(k, e) || off_size(v, e) || off_size(o, e) || off_size(lse, 4) ||
      off_size(k_length, 4) || ((uintptr_t)workspace & 255u))
    return LSTM_ERR_ALIGN;
  if (workspace_bytes < p.total_fwd) return LSTM_ERR_WORKSPACE;
  a.q = q; a.k = k; a.v = v; a.out = o; a.lse = lse;
  a.len = (const int32_t*)k_length;
  a.mask = (const uint8_t*)key_mask;
  a.splits = p.splits;
  a.part = (float*)((char*)workspace + p.off_part);
  a.part_ml = (float*)((char*)workspace + p.off_ml);
  const int64_t D = shape->D;
  a.whole = (whole_rows(q, a.qs, D, e) ? kWholeQ : 0) | (whole_rows(k, a.ks, D, e) ? kWholeK : 0) |
            (whole_rows(v, a.vs, D, e) ? kWholeV : 0) | (whole_rows(o, a.os, D, e) ? kWholeO : 0);
  p.dma = dma_rows(k, a.ks, D, e) && dma_rows(v, a.vs, D, e);
  return status(launch_attend_fwd(p, a, (hipStream_t)stream));
}

int lstm_attend_bwd(const lstm_attend_shape* shape, const void* dout, const void* q, const void* k, const void* v,
                    const void* k_length, const void* key_mask, const void* o, const float* lse, void* workspace,
                    size_t workspace_bytes, void* dq, void* dk, void* dv, void* stream) {
  AttendPlan p;
  const int rc = attend_plan(shape, true, &p);
  if (rc != LSTM_OK) return rc;
  AttendArgs a = attend_args(*shape);
  const bool rows = a.M > 0 && a.B > 0, keys = a.Tk > 0 && a.B > 0 && a.Hk > 0;
  if ((rows && (!dout || !q || !o || !lse || !dq || !workspace)) || (keys && (!k || !v || !dk || !dv)))
    return LSTM_ERR_NULL;
  const int64_t e = esize_of(p.dtype);
  if (off_size(dout, e) || off_size(q, e) || off_size(k, e) || off_size(v, e) || off_size(o, e) || off_size(lse, 4) ||
      off_size(k_length, 4) || off_size(dq, e) || off_size(dk, e) || off_size(dv, e) || ((uintptr_t)workspace & 255u))
    return LSTM_ERR_ALIGN;
  if (workspace_bytes < p.total_bwd) return LSTM_ERR_WORKSPACE;
  a.q = q; a.k = k; a.v = v; a.o = o; a.dout = dout; a.dq = dq; a.dk = dk; a.dv = dv;
  a.lse = const_cast<float*>(lse);
  a.stats = (float*)workspace;
  a.len = (const int32_t*)k_length;
  a.mask = (const uint8_t*)key_mask;
  const int64_t D = shape->D;
  a.whole = (whole_rows(q, a.qs, D, e) ? kWholeQ : 0) | (whole_rows(k, a.ks, D, e) ? kWholeK : 0) |
            (whole_rows(v, a.vs, D, e) ? kWholeV : 0) | (whole_rows(o, a.os, D, e) ? kWholeO : 0) |
            (whole_rows(dout, a.gs, D, e) ? kWholeG : 0) | (whole_rows(dq, a.dqs, D, e) ? kWholeDq : 0) |
            (whole_rows(dk, a.dks, D, e) ? kWholeDk : 0) | (whole_rows(dv, a.dvs, D, e) ? kWholeDv : 0);
  p.dma = dma_rows(q, a.qs, D, e) && dma_rows(k, a.ks, D, e) && dma_rows(v, a.vs, D, e) && dma_rows(dout, a.gs, D, e);
  return status(launch_attend_bwd(p, a, (hipStream_t)stream));
}

}  // extern "C"
