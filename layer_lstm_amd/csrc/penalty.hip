// penalty.hip -- penalties for repeated tokens, biases and masks on logits
// (gfx950).
//
// One pass: a work-group takes a slice of a row, counts the row's tokens so far
// that fall into the slice in LDS (whole numbers: the order of the additions
// does not matter), then reads, changes and writes the slice's logits, 16
// bytes a lane.  Logits read and written are the bound; the history is read
// once per slice from L2 (512 rows of 50000 bf16 logits, 2048 tokens each, bias
// and mask: 29 us of kernel, 139 MB with the histories' repeats, 4.8 TB/s).
#include "internal.hpp"
#include "model_internal.hpp"

namespace lstm {

// 32 KB of counts and 512 threads: four work-groups a compute unit, whose waves
// are all it holds (512 rows of 50000 bf16 logits, histories of up to 2048, bias
// and mask, us: 256 threads 47, slices of 4096 with 256 threads 39, of 16384 with
// 512 53, so 38).
constexpr int kPenThreads = 512;
constexpr int64_t kPenGroups = (((int64_t)1 << 32) - 1) / kPenThreads;  // of a launch, which has fewer than 2^32 threads
constexpr int kPenAhead = 2;         // 16-byte loads of logits a lane has under way
constexpr int64_t kPenSlice = 8192;  // logits of a work-group at most

// Fewer logits a work-group where that leaves four work-groups a compute unit.
void make_penalty_plan(int cus, PenaltyArgs* a) {
  int64_t slice = kPenSlice;
  const int64_t least = 256 * (a->dtype == LSTM_F32 ? 4 : 8);
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
  const T* x = (const T*)a.logits + n * a.ld + lo;
  T* y = (T*)a.out + n * a.ldo + lo;
  const float* bias = a.bias ? a.bias + n * a.ldb + lo : nullptr;
  const uint32_t* mask = a.mask ? a.mask + n * a.ldm + lo / 32 : nullptr;  // (lo: a multiple of 32)
  // the first logits, biases and mask bits are on their way while the history is counted
  u32x4_t ahead[kPenAhead], ahead_bias[kPenAhead][E / 4];
  uint32_t ahead_mask[kPenAhead];
  auto fetch = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kPenAhead; ++k) {
      const int i = i0 + (k * kPenThreads + tid) * E;
      if (i + E <= m) {
        ahead[k] = load16(x + i);
        if (bias) {
#pragma unroll
          for (int j = 0; j < E / 4; ++j) ahead_bias[k][j] = load16(bias + i + 4 * j);
        }
      }
      if (mask && i < m) ahead_mask[k] = mask[i / 32];
    }
  };
  fetch(0);
  RowPenalty r = {1.f, 0.f, 0.f};
  if constexpr (COUNT) {
    for (int i = tid * 4; i < (int)a.slice; i += kPenThreads * 4) *(u32x4_t*)(count + i) = u32x4_t{0, 0, 0, 0};
    __syncthreads();
    int64_t len = a.L;
    if (a.length) {
      const int64_t l = a.length[n];
      len = l < 0 ? 0 : l < a.L ? l : a.L;
    }
    const int64_t first = n * a.hn + tid * a.ht, step = kPenThreads * a.ht;
    auto tokens = [&](const auto* p) __attribute__((always_inline)) {
#pragma unroll 4
      for (int64_t t = tid; t < len; t += kPenThreads, p += step) {
        const int64_t id = (int64_t)*p - lo;
        if (id >= 0 && id < m) atomicAdd(count + id, 1u);
      }
    };
    if (a.id64) tokens((const int64_t*)a.history + first);
    else tokens((const int32_t*)a.history + first);
    if (a.repetition) r.rep = a.repetition[n];
    if (a.presence) r.presence = a.presence[n];
    if (a.frequency) r.frequency = a.frequency[n];
    __syncthreads();
  }
  for (int i0 = 0; i0 < m; i0 += kPenThreads * E * kPenAhead) {
    if (i0 > 0) fetch(i0);
#pragma unroll
    for (int k = 0; k < kPenAhead; ++k) {
      const int i = i0 + (k * kPenThreads + tid) * E;
      if (i >= m) break;
      float f[E];
      const bool whole = i + E <= m;
      if (whole) {
        unpack<T>(ahead[k], f);
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
            unpack<float>(ahead_bias[k][j / 4], g);
#pragma unroll
            for (int l = 0; l < 4; ++l) f[j + l] += g[l];
          }
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (i + j < m) f[j] += bias[i + j];
        }
      }
      if (mask) {
        const uint32_t bits = ahead_mask[k] >> (i % 32);
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
}

template <typename T>
static hipError_t penalty_of(const PenaltyArgs& a, hipStream_t s) {
  const bool count = a.L > 0 && (a.repetition || a.presence || a.frequency);
  const int64_t groups = a.N * a.slices;
  for (int64_t g = 0; g < groups; g += kPenGroups) {
    const unsigned n = (unsigned)(groups - g < kPenGroups ? groups - g : kPenGroups);
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
