// seq_api.hip -- the extern "C" entry points of the sequence-to-sequence
// operators (include/lstm.h): argument checks, then the launches.
#include "internal.hpp"
#include "seq_internal.hpp"

namespace lstm {

static bool dtype_ok(int d) { return d == LSTM_F32 || d == LSTM_BF16 || d == LSTM_F16; }
static bool id_ok(int t) { return t == LSTM_I32 || t == LSTM_I64; }
static bool off_size(const void* p, int64_t e) { return p && ((uintptr_t)p % (uintptr_t)e) != 0; }
static int status(hipError_t e) { return e == hipSuccess ? LSTM_OK : LSTM_ERR_LAUNCH; }
static int64_t esize_of(int dtype) { return dtype == LSTM_F32 ? 4 : 2; }

static int embed_plan(const lstm_embed_shape* s, EmbedPlan* p) {
  if (!s) return LSTM_ERR_NULL;
  if (s->N < 0 || s->V < 0 || s->D < 0 || s->ld_table < s->D || s->ld_out < s->D || s->padding < -1 ||
      s->padding >= (s->V > 0 ? s->V : 1))
    return LSTM_ERR_DIMS;
  if (!dtype_ok(s->dtype) || !id_ok(s->id_type)) return LSTM_ERR_DTYPE;
  const int64_t lim = (int64_t)1 << 26, far = (int64_t)1 << 36;  // row strides: offsets fit 63 bits
  if (s->N >= lim || s->V >= lim || s->D > ((int64_t)1 << 20) || s->ld_table >= far || s->ld_out >= far)
    return LSTM_ERR_UNSUPPORTED;
  int cus = 0;
  const int rc = device_cus(&cus);
  if (rc != LSTM_OK) return rc;
  make_embed_plan(*s, p);
  return LSTM_OK;
}

static int logprob_plan(const lstm_logprob_shape* s, LogprobPlan* p) {
  if (!s) return LSTM_ERR_NULL;
  if (s->N < 0 || s->V < 0 || s->ld < s->V || s->ld_grad < s->V || s->top < 0 || s->top > LSTM_MAX_TOP ||
      s->top > s->V || !(s->scale > 0.f) || s->scale > 3.0e38f)
    return LSTM_ERR_DIMS;
  if (!dtype_ok(s->dtype) || !id_ok(s->id_type)) return LSTM_ERR_DTYPE;
  const int64_t far = (int64_t)1 << 36;
  if (s->N >= ((int64_t)1 << 24) || s->V >= ((int64_t)1 << 30) || s->ld >= far || s->ld_grad >= far ||
      (s->V > 0 && s->N >= ((int64_t)1 << 37) / s->V))
    return LSTM_ERR_UNSUPPORTED;
  int cus = 0;
  const int rc = device_cus(&cus);
  if (rc != LSTM_OK) return rc;
  make_logprob_plan(*s, cus, p);
  return LSTM_OK;
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

}  // extern "C"
