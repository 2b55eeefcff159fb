// model_api.hip -- the extern "C" entry points of linear attention, the
// logits' penalties and the AdamW step (include/lstm.h): argument checks, then
// the launches.
#include <math.h>

#include "api_checks.hpp"
#include "attend_common.hpp"
#include "model_internal.hpp"

namespace lstm {

static int linattn_plan(const lstm_linattn_shape* s, bool bwd, LinPlan* p) {
  if (!s) return LSTM_ERR_NULL;
  if (s->T < 0 || s->B < 0 || s->Hq < 0 || s->Hk < 0 || s->D < 1 || s->Dv < 1 || (s->Hk == 0) != (s->Hq == 0) ||
      (s->Hk > 0 && s->Hq % s->Hk != 0) || !(fabsf(s->scale) <= 3.4e38f) ||
      !strides_ok(s->q) || !strides_ok(s->k) || !strides_ok(s->v) || !strides_ok(s->o) ||
      !disjoint(s->o, s->T, s->B, s->Hq, s->Dv))
    return LSTM_ERR_DIMS;
  if (bwd && (!strides_ok(s->dout) || !strides_ok(s->dq) || !strides_ok(s->dk) || !strides_ok(s->dv) ||
              !disjoint(s->dq, s->T, s->B, s->Hq, s->D) || !disjoint(s->dk, s->T, s->B, s->Hk, s->D) ||
              !disjoint(s->dv, s->T, s->B, s->Hk, s->Dv)))
    return LSTM_ERR_DIMS;
  if (!dtype_ok(s->dtype)) return LSTM_ERR_DTYPE;
  const int64_t wide = (int64_t)1 << 20;
  if (s->D > 256 || s->Dv > 256 || s->T >= ((int64_t)1 << 26) || s->B >= wide || s->Hq >= wide) return LSTM_ERR_UNSUPPORTED;
  // work-groups of any launch stay below 2^24, and below 2^16 along a grid's second axis
  if (s->B * s->Hq >= ((int64_t)1 << 18)) return LSTM_ERR_UNSUPPORTED;
  int cus = 0;
  const int rc = device_cus(&cus, nullptr);
  if (rc != LSTM_OK) return rc;
  make_linattn_plan(*s, cus, p);
  return LSTM_OK;
}

static LinArgs linattn_args(const lstm_linattn_shape& s, const float* log_decay, const void* length) {
  LinArgs a = {};
  a.T = s.T;
  a.B = (int)s.B;
  a.Hs = (int)s.Hk;
  a.log_decay = log_decay;
  a.len = (const int32_t*)length;
  a.scale = s.scale;
  a.segs = a.segs_of_launch = 1;
  return a;
}
struct Rows {
  const void* p;
  lstm_stride s;
  int64_t D;
};
// A run's tensors; *dma: all of them are whole aligned chunks that one descriptor reaches.
static LinRun linattn_run(const Rows& a, const Rows& k, const Rows& v, void* out, const lstm_stride& os, int64_t ga, int64_t gb,
                          int rev, int64_t e, int* dma) {
  LinRun r = {};
  r.a = a.p; r.k = k.p; r.v = v.p; r.out = out;
  r.as = a.s; r.ks = k.s; r.vs = v.s; r.os = os;
  r.DK = (int)k.D; r.DV = (int)v.D;
  r.ga = (int)ga; r.gb = (int)gb;
  r.rev = rev;
  r.whole = (whole_rows(a.p, a.s, a.D, e) ? kWholeQ : 0) | (whole_rows(k.p, k.s, k.D, e) ? kWholeK : 0) |
            (whole_rows(v.p, v.s, v.D, e) ? kWholeV : 0) | (whole_rows(out, os, v.D, e) ? kWholeO : 0);
  auto reach = [&](const Rows& x) { return whole_rows(x.p, x.s, x.D, e) && x.s.t >= x.D && x.s.t * e < ((int64_t)1 << 31) / 64; };
  *dma = reach(a) && reach(k) && reach(v);
  return r;
}

static int penalty_plan(const lstm_penalty_shape* s, PenaltyArgs* a) {
  if (!s) return LSTM_ERR_NULL;
  if (s->N < 0 || s->V < 0 || s->L < 0 || s->ld < s->V || s->ld_out < s->V || s->history_n < 0 || s->history_t < 0 ||
      s->ld_bias < 0 || s->ld_mask < 0)
    return LSTM_ERR_DIMS;
  if (!dtype_ok(s->dtype) || !id_ok(s->id_type)) return LSTM_ERR_DTYPE;
  const int64_t far = (int64_t)1 << 36;
  if (s->N >= ((int64_t)1 << 24) || s->V >= ((int64_t)1 << 30) || s->L >= ((int64_t)1 << 31) || s->ld >= far ||
      s->ld_out >= far || s->history_n >= far || s->history_t >= ((int64_t)1 << 31) || s->ld_bias >= far ||
      s->ld_mask >= far || (s->V > 0 && s->N >= ((int64_t)1 << 37) / s->V))
    return LSTM_ERR_UNSUPPORTED;
  int cus = 0;
  const int rc = device_cus(&cus, nullptr);
  if (rc != LSTM_OK) return rc;
  *a = {};
  a->N = s->N; a->V = s->V; a->ld = s->ld; a->ldo = s->ld_out;
  a->L = s->L; a->hn = s->history_n; a->ht = s->history_t;
  a->ldb = s->ld_bias; a->ldm = s->ld_mask;
  a->dtype = s->dtype; a->id64 = s->id_type == LSTM_I64;
  make_penalty_plan(cus, a);
  return LSTM_OK;
}

// Rows of logits and out that are neither the same nor apart: in memory that is
// not the other's, or other columns of the same rows.
static bool penalty_overlap(const PenaltyArgs& a, const void* logits, const void* out, int64_t e) {
  if (a.N == 0 || a.V == 0 || (logits == out && a.ld == a.ldo)) return false;
  const int64_t x = (int64_t)(uintptr_t)logits, y = (int64_t)(uintptr_t)out;
  if (y >= x + ((a.N - 1) * a.ld + a.V) * e || x >= y + ((a.N - 1) * a.ldo + a.V) * e) return false;
  if (a.ld != a.ldo || a.N == 1) return true;
  const int64_t row = a.ld * e, d = ((y - x) % row + row) % row;
  return d < a.V * e || d > row - a.V * e;
}

// The step's or the norm's arguments; the norm reads grad and n alone.
static int adamw_plan(const lstm_adamw_shape* s, const lstm_adamw_tensor* t, int64_t count, bool step, bool control,
                      AdamwPlan* p) {
  if (!s || (count > 0 && !t)) return LSTM_ERR_NULL;
  if (count < 0 || !(s->lr >= 0 && s->lr < HUGE_VAL) || !(s->eps >= 0 && s->eps < HUGE_VAL) ||
      !(s->beta1 >= 0 && s->beta1 < 1) || !(s->beta2 >= 0 && s->beta2 < 1) || (step && !control && s->step < 1))
    return LSTM_ERR_DIMS;
  for (int64_t k = 0; k < count; ++k)
    if (t[k].n < 0 || (step && !(t[k].weight_decay >= 0 && t[k].weight_decay < HUGE_VAL))) return LSTM_ERR_DIMS;
  if (!dtype_ok(s->dtype) || (s->bits != 32 && s->bits != 8)) return LSTM_ERR_DTYPE;
  if (count >= ((int64_t)1 << 20)) return LSTM_ERR_UNSUPPORTED;
  int64_t all = 0;
  for (int64_t k = 0; k < count; ++k) {
    if (t[k].n >= ((int64_t)1 << 40)) return LSTM_ERR_UNSUPPORTED;
    all += t[k].n;
    if (all >= ((int64_t)1 << 40)) return LSTM_ERR_UNSUPPORTED;
  }
  const int64_t e = esize_of(s->dtype), se = s->bits / 8;
  for (int64_t k = 0; k < count; ++k) {
    if (t[k].n == 0) continue;
    if (!t[k].grad || (step && (!t[k].param || !t[k].m || !t[k].v || (s->bits == 8 && (!t[k].m_scale || !t[k].v_scale)))))
      return LSTM_ERR_NULL;
  }
  for (int64_t k = 0; k < count; ++k) {
    if (t[k].n == 0) continue;
    if (off_size(t[k].grad, e) || (step && (off_size(t[k].param, e) || off_size(t[k].master, 4) || off_size(t[k].m, se) ||
                                            off_size(t[k].v, se) || off_size(t[k].m_scale, 4) || off_size(t[k].v_scale, 4))))
      return LSTM_ERR_ALIGN;
  }
  int cus = 0;
  const int rc = device_cus(&cus, nullptr);
  if (rc != LSTM_OK) return rc;
  *p = {s->lr, s->beta1, s->beta2, s->eps, s->step, s->dtype, s->bits};
  return LSTM_OK;
}
static size_t norm_bytes(const lstm_adamw_tensor* t, int64_t count) {
  size_t n = 0;
  for (int64_t k = 0; k < count; ++k) n += (size_t)((t[k].n + kNormChunk - 1) / kNormChunk);
  return align256_seq(n * 8);
}

}  // namespace lstm

using namespace lstm;

extern "C" {

int lstm_linattn_query(const lstm_linattn_shape* shape, size_t* fwd_bytes, size_t* bwd_bytes) {
  if (!fwd_bytes || !bwd_bytes) return LSTM_ERR_NULL;
  LinPlan p;
  const int rc = linattn_plan(shape, false, &p);
  if (rc != LSTM_OK) return rc;
  *fwd_bytes = p.total_fwd;
  *bwd_bytes = p.total_bwd;
  return LSTM_OK;
}

int lstm_linattn_fwd(const lstm_linattn_shape* shape, const void* q, const void* k, const void* v,
                     const float* log_decay, const void* length, const float* state, void* workspace,
                     size_t workspace_bytes, void* o, float* state_out, void* stream) {
  LinPlan p;
  const int rc = linattn_plan(shape, false, &p);
  if (rc != LSTM_OK) return rc;
  const lstm_linattn_shape& s = *shape;
  const bool heads = s.B > 0 && s.Hk > 0, rows = heads && s.T > 0;
  if ((heads && !log_decay) || (rows && (!q || !k || !v || !o || (p.total_fwd > 0 && !workspace)))) return LSTM_ERR_NULL;
  const int64_t e = esize_of(p.dtype);
  if (off_size(q, e) || off_size(k, e) || off_size(v, e) || off_size(o, e) || off_size(log_decay, 4) || off_size(length, 4) ||
      off_size(state, 4) || off_size(state_out, 4) || ((uintptr_t)workspace & 255u))
    return LSTM_ERR_ALIGN;
  if (rows && workspace_bytes < p.total_fwd) return LSTM_ERR_WORKSPACE;
  if ((state && state == state_out && !p.step) || (rows && (o == q || o == k || o == v))) return LSTM_ERR_DIMS;
  if (!heads) return LSTM_OK;
  LinArgs a = linattn_args(s, log_decay, length);
  int dma;
  a.runs = 1;
  a.run[0] = linattn_run({q, s.q, s.D}, {k, s.k, s.D}, {v, s.v, s.Dv}, o, s.o, s.Hq / s.Hk, 1, 0, e, &dma);
  LinRun& r = a.run[0];
  r.s_in = state; r.s_out = state_out;
  r.s_dk = s.Dv; r.s_dv = 1;
  r.seg = (float*)workspace;
  if (p.step) return status(launch_linattn_step(p, a, (hipStream_t)stream));
  return status(launch_linattn(p, p.fwd, a, &dma, (hipStream_t)stream));
}

int lstm_linattn_bwd(const lstm_linattn_shape* shape, const void* dout, const void* q, const void* k, const void* v,
                     const float* log_decay, const void* length, const float* state, const float* dstate,
                     void* workspace, size_t workspace_bytes, void* dq, void* dk, void* dv, float* dstate0,
                     void* stream) {
  LinPlan p;
  const int rc = linattn_plan(shape, true, &p);
  if (rc != LSTM_OK) return rc;
  const lstm_linattn_shape& s = *shape;
  const bool heads = s.B > 0 && s.Hk > 0, rows = heads && s.T > 0;
  if ((heads && !log_decay) ||
      (rows && (!dout || !q || !k || !v || !dq || !dk || !dv || (p.total_bwd > 0 && !workspace))))
    return LSTM_ERR_NULL;
  const int64_t e = esize_of(p.dtype);
  if (off_size(dout, e) || off_size(q, e) || off_size(k, e) || off_size(v, e) || off_size(dq, e) || off_size(dk, e) ||
      off_size(dv, e) || off_size(log_decay, 4) || off_size(length, 4) || off_size(state, 4) || off_size(dstate, 4) ||
      off_size(dstate0, 4) || ((uintptr_t)workspace & 255u))
    return LSTM_ERR_ALIGN;
  if (rows && workspace_bytes < p.total_bwd) return LSTM_ERR_WORKSPACE;
  if (dstate && dstate == dstate0) return LSTM_ERR_DIMS;
  for (const void* in : {dout, q, k, v})
    if (rows && (in == dq || in == dk || in == dv)) return LSTM_ERR_DIMS;
  if (!heads) return LSTM_OK;
  LinArgs a = linattn_args(s, log_decay, length);
  const int64_t G = s.Hq / s.Hk;
  const Rows rq = {q, s.q, s.D}, rk = {k, s.k, s.D}, rv = {v, s.v, s.Dv}, rg = {dout, s.dout, s.Dv};
  int dma[3];
  a.runs = 3;
  a.run[0] = linattn_run(rg, rv, rk, dq, s.dq, G, 1, 0, e, &dma[0]);   // state S^T
  a.run[1] = linattn_run(rv, rg, rq, dk, s.dk, 1, G, 1, e, &dma[1]);   // state R^T
  a.run[2] = linattn_run(rk, rq, rg, dv, s.dv, 1, G, 1, e, &dma[2]);   // state R
  for (int i = 0; i < 3; ++i) {
    LinRun& r = a.run[i];
    r.s_in = i == 0 ? state : dstate;
    r.s_dk = i == 2 ? s.Dv : 1;
    r.s_dv = i == 2 ? 1 : s.Dv;
    r.seg = (float*)((char*)workspace + i * p.seg_bytes);
  }
  a.run[2].s_out = dstate0;
  return status(launch_linattn(p, p.bwd, a, dma, (hipStream_t)stream));
}

int lstm_penalty(const lstm_penalty_shape* shape, const void* logits, const void* history, const void* history_length,
                 const float* repetition, const float* presence, const float* frequency, const float* bias,
                 const uint32_t* mask, void* out, void* stream) {
  PenaltyArgs a;
  const int rc = penalty_plan(shape, &a);
  if (rc != LSTM_OK) return rc;
  if ((bias && a.ldb != 0 && a.ldb < a.V) || (mask && a.ldm < (a.V + 31) / 32) || (out && out == logits && a.ld != a.ldo))
    return LSTM_ERR_DIMS;
  const bool counts = a.L > 0 && (repetition || presence || frequency);
  if (a.N > 0 && a.V > 0 && (!logits || !out || (counts && !history))) return LSTM_ERR_NULL;
  const int64_t e = esize_of(a.dtype);
  if (off_size(logits, e) || off_size(out, e) || off_size(history, a.id64 ? 8 : 4) || off_size(history_length, 4) ||
      off_size(repetition, 4) || off_size(presence, 4) || off_size(frequency, 4) || off_size(bias, 4) || off_size(mask, 4))
    return LSTM_ERR_ALIGN;
  if (penalty_overlap(a, logits, out, e)) return LSTM_ERR_DIMS;
  a.logits = logits; a.history = history; a.length = (const int32_t*)history_length;
  a.repetition = repetition; a.presence = presence; a.frequency = frequency;
  a.bias = bias; a.mask = mask; a.out = out;
  return status(launch_penalty(a, (hipStream_t)stream));
}

int lstm_adamw_query(const lstm_adamw_shape* shape, const lstm_adamw_tensor* tensors, int64_t count,
                     size_t* workspace_bytes) {
  if (!workspace_bytes || !shape || (count > 0 && !tensors)) return LSTM_ERR_NULL;
  if (count < 0) return LSTM_ERR_DIMS;
  for (int64_t k = 0; k < count; ++k)
    if (tensors[k].n < 0) return LSTM_ERR_DIMS;
  if (count >= ((int64_t)1 << 20)) return LSTM_ERR_UNSUPPORTED;
  for (int64_t k = 0; k < count; ++k)
    if (tensors[k].n >= ((int64_t)1 << 40)) return LSTM_ERR_UNSUPPORTED;
  *workspace_bytes = norm_bytes(tensors, count);
  return LSTM_OK;
}

int lstm_adamw_norm(const lstm_adamw_shape* shape, const lstm_adamw_tensor* tensors, int64_t count, double max_norm,
                    double unscale, void* workspace, size_t workspace_bytes, lstm_adamw_control* control, void* stream) {
  AdamwPlan p;
  if (!(max_norm > 0) || !(unscale > 0 && unscale < HUGE_VAL)) return shape ? LSTM_ERR_DIMS : LSTM_ERR_NULL;
  const int rc = adamw_plan(shape, tensors, count, false, true, &p);
  if (rc != LSTM_OK) return rc;
  const size_t need = norm_bytes(tensors, count);
  if (!control || (need > 0 && !workspace)) return LSTM_ERR_NULL;
  if (((uintptr_t)workspace & 255u) || off_size(control, 8)) return LSTM_ERR_ALIGN;
  if (workspace_bytes < need) return LSTM_ERR_WORKSPACE;
  return status(launch_adamw_norm(p, tensors, count, max_norm, unscale, (double*)workspace, control, (hipStream_t)stream));
}

int lstm_adamw_step(const lstm_adamw_shape* shape, const lstm_adamw_tensor* tensors, int64_t count,
                    const lstm_adamw_control* control, void* stream) {
  AdamwPlan p;
  const int rc = adamw_plan(shape, tensors, count, true, control != nullptr, &p);
  if (rc != LSTM_OK) return rc;
  if (off_size(control, 8)) return LSTM_ERR_ALIGN;
  return status(launch_adamw_step(p, tensors, count, control, (hipStream_t)stream));
}

}  // extern "C"
