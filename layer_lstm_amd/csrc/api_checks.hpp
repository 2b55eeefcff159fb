// api_checks.hpp -- argument checks that the operators' entry points share.
#pragma once
#include "internal.hpp"
#include "seq_internal.hpp"

namespace lstm {

static inline bool dtype_ok(int d) { return d == LSTM_F32 || d == LSTM_BF16 || d == LSTM_F16; }
static inline bool id_ok(int t) { return t == LSTM_I32 || t == LSTM_I64; }
// a softmax's scale: scale log2 e is a positive number
static inline bool scale_ok(float s) { return s > 0.f && s <= 2.3e38f; }
static inline bool off_size(const void* p, int64_t e) { return p && ((uintptr_t)p % (uintptr_t)e) != 0; }
static inline int status(hipError_t e) { return e == hipSuccess ? LSTM_OK : LSTM_ERR_LAUNCH; }
static inline int64_t esize_of(int dtype) { return dtype == LSTM_F32 ? 4 : 2; }

// A tensor of [T][B][H] rows of D values whose rows do not overlap.
static inline bool disjoint(const lstm_stride& s, int64_t T, int64_t B, int64_t H, int64_t D) {
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
static inline bool strides_ok(const lstm_stride& s) {
  const int64_t far = (int64_t)1 << 36;
  return s.t >= 0 && s.b >= 0 && s.h >= 0 && s.t < far && s.b < far && s.h < far;
}
// whole aligned 16-byte chunks in every row
static inline bool whole_rows(const void* p, const lstm_stride& s, int64_t D, int64_t e) {
  return aligned16(p) && (D * e) % 16 == 0 && (s.t * e) % 16 == 0 && (s.b * e) % 16 == 0 && (s.h * e) % 16 == 0;
}

}  // namespace lstm
