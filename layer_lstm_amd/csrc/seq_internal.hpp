// seq_internal.hpp -- what the sequence-to-sequence operators share: packed
// 16-byte rows, and the launchers seq_api.hip calls.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "device_common.hpp"
#include "lstm.h"

namespace lstm {

// Compute units (and index) of the current device; LSTM_ERR_DEVICE if it is
// not a gfx950 (lstm_api.hip).
int device_cus(int* cus, int* devp);

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Elements of 16 bytes of storage type T.
template <typename T> constexpr int vec_of() { return 16 / (int)sizeof(T); }

// Two fp32 values to a word of two 16-bit values, nearest even
// (v_cvt_pk_bf16_f32 / v_cvt_f16_f32; NaN stays NaN).
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
// The value as an fp32 register: a product is rounded to fp32 here and not
// folded into its conversion to fp16 (v_fma_mixlo_f16 rounds the exact
// product), so that every path of an operator gives the same bits.
__device__ __forceinline__ float as_f32(float v) {
  asm("" : "+v"(v));
  return v;
}
template <> __device__ __forceinline__ uint32_t pack2<bf16_t>(float a, float b) {
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
template <> __device__ __forceinline__ uint32_t pack2<f16_t>(float a, float b) {
  const f32x2_t v = {as_f32(a), as_f32(b)};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}

// 16 bytes of storage <-> fp32 values.
template <typename T>
__device__ __forceinline__ void unpack(u32x4_t v, float* f) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = f_of_bits16<T>(v[i] & 0xffffu);
      f[2 * i + 1] = f_of_bits16<T>(v[i] >> 16);
    }
  }
}
template <typename T>
__device__ __forceinline__ u32x4_t pack(const float* f) {
  u32x4_t v;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
  }
  return v;
}

// A launch has fewer than 2^32 threads: work-groups of 256 that one may have.
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;

static inline size_t align256_seq(size_t v) { return (v + 255) & ~(size_t)255; }
static inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// ---- embed.hip ----
// Workspace of the table's gradient: the tokens sorted by id (two buffers of
// (id, position) pairs), the digit counts of the sort's blocks, each row's
// range of sorted positions, and the sums of whole chunks of one id.
struct EmbedPlan {
  int64_t N, V, D, ldt, ldo, padding;
  float scale;
  int dtype, id64;
  int bits, passes, digit;  // of the sort: bits of an id, passes of `digit` bits
  int few;                  // the gradient in one launch, without a workspace
  int rounds, blocks;       // of the sort: blocks of 1024 * rounds tokens
  size_t off_pair0, off_pair1, off_hist, off_seg, off_part, total;
};
void make_embed_plan(const lstm_embed_shape& s, EmbedPlan* p);
hipError_t launch_embed_fwd(const EmbedPlan& p, const void* ids, const void* table, void* out, hipStream_t s);
hipError_t launch_embed_bwd(const EmbedPlan& p, const void* ids, const void* dout, char* ws, void* dtable,
                            hipStream_t s);

// ---- logprob.hip ----
struct LogprobPlan {
  int64_t N, V, ld, ldg;
  float scale;
  int top, dtype, id64;
  int parts;        // waves a row of the forward is split over
  int64_t part;     // logits of each (a multiple of one round of a wave's loads)
  size_t off_key, off_sum, total;
};
void make_logprob_plan(const lstm_logprob_shape& s, int cus, LogprobPlan* p);
hipError_t launch_logprob_fwd(const LogprobPlan& p, const void* logits, const void* targets, char* ws, float* record,
                              float* lse, float* logp, float* entropy, float* top_logp, void* top_ids, hipStream_t s);
hipError_t launch_logprob_bwd(const LogprobPlan& p, const void* logits, const void* targets, const float* record,
                              const float* entropy, const void* top_ids, const float* dlogp, const float* dentropy,
                              const float* dtop, void* dlogits, hipStream_t s);

// ---- attend.hip, attend_bwd.hpp ----
struct AttendArgs;
struct AttendPlan {
  int dtype, DP;    // DP: the head size the kernels run with
  int dma;          // rows are whole aligned 16-byte chunks that do not overlap
  int step;         // forward by attend_step_kernel,
  int splits;       //   the keys of a row tile split over this many work-groups
  int few_rows, few_keys;  // backward: dq, dk and dv by the kernels that split the sums over waves
  int row_tiles32;  // tiles of 32 rows per (sequence, key head)
  size_t off_part, off_ml, total_fwd, total_bwd;
};
void make_attend_plan(const lstm_attend_shape& s, int cus, AttendPlan* p);
hipError_t launch_attend_fwd(const AttendPlan& p, const AttendArgs& a, hipStream_t s);
hipError_t launch_attend_bwd(const AttendPlan& p, const AttendArgs& a, hipStream_t s);
hipError_t launch_attend_bwd_f32(const AttendPlan& p, const AttendArgs& a, hipStream_t s);
hipError_t launch_attend_bwd_bf16(const AttendPlan& p, const AttendArgs& a, hipStream_t s);
hipError_t launch_attend_bwd_f16(const AttendPlan& p, const AttendArgs& a, hipStream_t s);

}  // namespace lstm
