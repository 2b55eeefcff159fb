// penalty.hip -- penalties for repeated tokens, biases and masks on logits
// (gfx950).
//
// One pass: a work-group takes a slice of a row, counts the row's tokens so far
// that fall into the slice in LDS (whole numbers: the order of the additions
// does not matter), then reads, changes and writes the slice's logits, 16
// bytes a lane.  Logits read and written are the bound; the history is read
// once per slice from L2.
#include "internal.hpp"
#include "model_internal.hpp"

namespace lstm {

constexpr int kPenThreads = 256;
constexpr int64_t kPenSlice = 8192;  // logits of a work-group at most: 32 KB of counts

// As many logits a work-group as leave four work-groups a compute unit.
void make_penalty_plan(int cus, PenaltyArgs* a) {
  int64_t slice = kPenSlice;
  const int64_t least = kPenThreads * (a->dtype == LSTM_F32 ? 4 : 8);
  while (slice > least && a->N * ((a->V + slice - 1) / slice) < 4 * (int64_t)cus) slice /= 2;
  a->slice = slice;
  a->slices = (int)((a->V + slice - 1) / slice);
}

// 16 bytes at any alignment of the element.
__device__ __forceinline__ u32x4_t load16(const void* p) {
  u32x4_t v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ void store16(void* p, u32x4_t v) { __builtin_memcpy(p, &v, 16); }

struct RowPenalty {
  float rep, presence, frequency;
};
__device__ __forceinline__ float penalised(float x, uint32_t c, const RowPenalty& r) {
#pragma clang fp contract(off)
  if (c == 0) return x;
  x = x > 0.f ? x / r.rep : x * r.rep;
  return x - (r.presence + r.frequency * (float)c);
}

template <typename T, bool COUNT>
__global__ void __launch_bounds__(kPenThreads) penalty_kernel(PenaltyArgs a, int64_t group0) {
  constexpr int E = vec_of<T>();
  extern __shared__ __attribute__((aligned(16))) uint32_t count[];
  const int64_t unit = group0 + blockIdx.x, n = unit / a.slices, lo = (unit - n * a.slices) * a.slice;
  const int tid = threadIdx.x;
  const int m = (int)(lo + a.slice < a.V ? a.slice : a.V - lo);  // logits of the slice
  RowPenalty r = {1.f, 0.f, 0.f};
  if constexpr (COUNT) {
    for (int i = tid * 4; i < (int)a.slice; i += kPenThreads * 4) *(u32x4_t*)(count + i) = u32x4_t{0, 0, 0, 0};
    __syncthreads();
    int64_t len = a.L;
    if (a.length) {
      const int64_t l = a.length[n];
      len = l < 0 ? 0 : l < a.L ? l : a.L;
    }
    for (int64_t t = tid; t < len; t += kPenThreads) {
      const int64_t at = n * a.hn + t * a.ht;
      const int64_t id = (a.id64 ? ((const int64_t*)a.history)[at] : (int64_t)((const int32_t*)a.history)[at]) - lo;
      if (id >= 0 && id < m) atomicAdd(count + id, 1u);
    }
    if (a.repetition) r.rep = a.repetition[n];
    if (a.presence) r.presence = a.presence[n];
    if (a.frequency) r.frequency = a.frequency[n];
    __syncthreads();
  }
  const T* x = (const T*)a.logits + n * a.ld + lo;
  T* y = (T*)a.out + n * a.ldo + lo;
  const float* bias = a.bias ? a.bias + n * a.ldb + lo : nullptr;
  const uint32_t* mask = a.mask ? a.mask + n * a.ldm + lo / 32 : nullptr;  // (lo: a multiple of 32)
  for (int i = tid * E; i < m; i += kPenThreads * E) {
    float f[E];
    const bool whole = i + E <= m;
    if (whole) {
      unpack<T>(load16(x + i), f);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) f[j] = i + j < m ? Elem<T>::load(x + i + j) : 0.f;
    }
    if constexpr (COUNT) {
      uint32_t c[E], any = 0;
#pragma unroll
      for (int j = 0; j < E; j += 4) *(u32x4_t*)(c + j) = *(const u32x4_t*)(count + i + j);
#pragma unroll
      for (int j = 0; j < E; ++j) any |= c[j];
      if (any) {
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = penalised(f[j], c[j], r);
      }
    }
    if (bias) {
      if (whole) {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
          float g[4];
          unpack<float>(load16(bias + i + j), g);
#pragma unroll
          for (int k = 0; k < 4; ++k) f[j + k] += g[k];
        }
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (i + j < m) f[j] += bias[i + j];
      }
    }
    if (mask) {
      const uint32_t bits = mask[i / 32] >> (i % 32);
#pragma unroll
      for (int j = 0; j < E; ++j) f[j] = (bits >> j) & 1 ? f[j] : -INFINITY;
    }
    if (whole) {
      store16(y + i, pack<T>(f));
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (i + j < m) y[i + j] = Elem<T>::from_f(f[j]);
    }
  }
}

template <typename T>
static hipError_t penalty_of(const PenaltyArgs& a, hipStream_t s) {
  const bool count = a.L > 0 && (a.repetition || a.presence || a.frequency);
  const int64_t groups = a.N * a.slices;
  for (int64_t g = 0; g < groups; g += kMaxGroups) {
    const unsigned n = (unsigned)(groups - g < kMaxGroups ? groups - g : kMaxGroups);
    Timed timed(11, s);
    if (count) penalty_kernel<T, true><<<dim3(n), kPenThreads, (size_t)a.slice * 4, s>>>(a, g);
    else penalty_kernel<T, false><<<dim3(n), kPenThreads, 0, s>>>(a, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_penalty(const PenaltyArgs& a, hipStream_t s) {
  if (a.N == 0 || a.V == 0) return hipSuccess;
  if (a.dtype == LSTM_F32) return penalty_of<float>(a, s);
  if (a.dtype == LSTM_BF16) return penalty_of<bf16_t>(a, s);
  return penalty_of<f16_t>(a, s);
}

}  // namespace lstm
