// logprob.hip -- log probabilities of given tokens, entropy, best
// alternatives, and the logits' gradient (gfx950).
//
// One pass over a row keeps, per lane, s = sum 2^y and t = sum 2^y y of
// y = (x - m) scale log2(e) against a reference m of the wave, so that
//   lse = scale m + ln 2 log2 s,   entropy = ln 2 (log2 s - t / s),
//   log p = scale (x - m) - ln 2 log2 s,
// the last without the rounding of lse, which for logits of large magnitude
// (a row of the type's lowest value, say) would be all of the result: the
// gradient therefore reads m and ln s (the record) and not lse.
// The reference need not be the running maximum: any m that no logit passes
// by more than kSlack keeps 2^y in range and costs no precision (s and t are
// floating point), so it moves only when a logit does pass it, which after
// the first few vectors of a row is rare, and the sums are rescaled then.
//
// The alternatives are kept as a list sorted across the lanes of a wave: a
// 64-bit key per lane, the logit in an order-preserving form above the
// complement of its id, so that no two keys are equal and a tie goes to the
// lower id.  A vector whose largest logit does not reach the list's entry
// `top` is passed over with one comparison.
#include <type_traits>

#include "internal.hpp"
#include "seq_internal.hpp"

namespace lstm {

constexpr int kLpThreads = 256, kLpWaves = 4;
constexpr int kMaxParts = 64;   // a row's parts are joined by the lanes of one wave
constexpr float kSlack = 16.f;  // how far (in powers of two) a logit may pass the reference

void make_logprob_plan(const lstm_logprob_shape& s, int cus, LogprobPlan* p) {
  p->N = s.N; p->V = s.V; p->ld = s.ld; p->ldg = s.ld_grad;
  p->scale = s.scale; p->top = s.top; p->dtype = s.dtype; p->id64 = s.id_type == LSTM_I64;
  // a work-group per row; rows too few for four work-groups a compute unit
  // are split, down to one vector per thread
  const int64_t step = (int64_t)kLpThreads * (s.dtype == LSTM_F32 ? 4 : 8);
  int64_t parts = 1;
  if (s.N > 0 && s.N < 4 * (int64_t)cus) parts = 4 * (int64_t)cus / s.N;
  if (parts > kMaxParts) parts = kMaxParts;
  int64_t steps = (s.V + step - 1) / step;  // of a row
  if (steps < 1) steps = 1;
  const int64_t each = (steps + parts - 1) / parts;
  p->part = each * step;
  p->parts = (int)((steps + each - 1) / each);
  size_t off = 0;
  p->off_key = p->off_sum = 0;
  if (p->parts > 1) {
    p->off_key = off; off += align256_seq((size_t)s.N * p->parts * s.top * 8);
    p->off_sum = off; off += align256_seq((size_t)s.N * p->parts * 16);
  }
  p->total = off;
}

// A logit as an unsigned integer of the same order (-0 taken as +0).
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ (uint32_t)(((int32_t)u >> 31) | (int32_t)0x80000000);
}
__device__ __forceinline__ float from_order(uint32_t o) {
  return __uint_as_float(o ^ ((o & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sums against a reference, moved to another reference.
struct RowSums {
  float m, s, t;  // m = -inf: nothing but -inf so far (s = t = 0, or NaN)
  __device__ __forceinline__ float ref() const { return m == -INFINITY ? 0.f : m; }
  __device__ __forceinline__ void move(float to, float c2) {
    if (m != -INFINITY && to != m) {
      const float d = (to - m) * c2, r = __builtin_amdgcn_exp2f(-d);
      t = r == 0.f ? s * 0.f : (t - d * s) * r;
      s *= r;
    }
    m = to;
  }
};

// The list: lane i holds the i-th largest key so far (0: none).
struct TopList {
  uint32_t hi, lo;    // this lane's key
  uint32_t thi, tlo;  // key `top` - 1, which a key has to pass
  float tval;         // its logit
  bool full;
  __device__ __forceinline__ void clear() { hi = lo = thi = tlo = 0; tval = -INFINITY; full = false; }
  // true in the lanes whose vector may hold a key to insert
  __device__ __forceinline__ bool wants(float vmax) const { return !full || vmax >= tval; }
  __device__ __forceinline__ void insert(uint32_t chi, uint32_t clo, int top, int lane) {
    uint64_t cand = __ballot(chi > thi || (chi == thi && clo > tlo));
    while (cand) {
      const int l = __builtin_ctzll(cand);
      const uint32_t a = __builtin_amdgcn_readlane(chi, l), b = __builtin_amdgcn_readlane(clo, l);
      const int at = __popcll(__ballot(hi > a || (hi == a && lo > b)));
      const uint32_t shi = __shfl_up(hi, 1), slo = __shfl_up(lo, 1);
      hi = lane < at ? hi : lane == at ? a : shi;
      lo = lane < at ? lo : lane == at ? b : slo;
      thi = __builtin_amdgcn_readlane(hi, top - 1);
      tlo = __builtin_amdgcn_readlane(lo, top - 1);
      cand &= ~((uint64_t)2 << l) + 1;  // the lanes after l
      cand &= __ballot(chi > thi || (chi == thi && clo > tlo));
    }
    full = thi != 0 || tlo != 0;
    tval = from_order(thi);
  }
};

struct LogprobOut {
  float *record, *lse, *logp, *entropy, *top_logp;
  void* top_ids;
  int id64;
};

__device__ __forceinline__ int64_t id_at(const void* ids, int64_t i, int id64) {
  return id64 ? ((const int64_t*)ids)[i] : (int64_t)((const int32_t*)ids)[i];
}

// (m, ls): a row's record
__device__ __forceinline__ float log_prob(float x, float scale, float m, float ls) {
  return m == -INFINITY ? -INFINITY : (x - m) * scale - ls;
}

// A row's results from its sums; called by every thread of the group that
// writes them, `key` the sorted list.
template <typename T>
__device__ __forceinline__ void finish_row(const LogprobOut& o, int64_t n, const T* row, const void* targets, int64_t V,
                                           float scale, int top, RowSums r, const uint64_t* key, int tid) {
  const float l2 = log2f(r.s), ls = kLn2 * l2;
  if (tid == 0) {
    o.record[2 * n] = r.m;
    o.record[2 * n + 1] = ls;
    if (o.lse) o.lse[n] = r.m * scale + ls;
    if (o.entropy) o.entropy[n] = r.m == -INFINITY && r.s == 0.f ? 0.f : kLn2 * (l2 - r.t / r.s);
  }
  if (tid == 32 && o.logp) {
    const int64_t id = id_at(targets, n, o.id64);
    o.logp[n] = id >= 0 && id < V ? log_prob(Elem<T>::load(row + id), scale, r.m, ls) : 0.f;
  }
  if (tid < top) {
    const uint64_t k = key[tid];
    const uint32_t id = ~(uint32_t)k;
    o.top_logp[n * top + tid] = log_prob(from_order((uint32_t)(k >> 32)), scale, r.m, ls);
    if (o.id64) ((int64_t*)o.top_ids)[n * top + tid] = id;
    else ((int32_t*)o.top_ids)[n * top + tid] = (int32_t)id;
  }
}

// A work-group per (row, part).
template <typename T, bool TOP>
__global__ void __launch_bounds__(kLpThreads) logprob_fwd_kernel(const T* logits, const void* targets, int64_t V,
                                                                 int64_t ld, float scale, int top, int parts,
                                                                 int64_t part, LogprobOut out, uint64_t* wkey,
                                                                 f32x4_t* wsum) {
  constexpr int E = vec_of<T>();
  constexpr int U = 4;  // vectors a thread has in flight
  __shared__ RowSums sums[kLpWaves];
  __shared__ uint64_t keys[kLpWaves * LSTM_MAX_TOP], best[LSTM_MAX_TOP];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t n = blockIdx.x / parts;
  const int pt = (int)(blockIdx.x - n * parts);
  const T* row = logits + n * ld;
  const int64_t lo = (int64_t)pt * part, hi = lo + part < V ? lo + part : V;
  const float c2 = scale * kLog2e, slack = kSlack / c2;

  RowSums r = {-INFINITY, 0.f, 0.f};
  TopList list;
  list.clear();
  // C logits of this lane at ids id0 .. (valid: the lane has any)
  auto take = [&](const float* f, auto C, int64_t id0, bool valid) {
    constexpr int c = decltype(C)::value;
    float vm = f[0];
#pragma unroll
    for (int j = 1; j < c; ++j) vm = fmaxf(vm, f[j]);
    if (__ballot(vm > r.m + slack || (vm > r.m && r.m == -INFINITY))) {
      const float to = wave_max(vm);
      r.move(to, c2);
    }
    const float m = r.ref();
#pragma unroll
    for (int j = 0; j < c; ++j) {
      const float y = (f[j] - m) * c2, e = __builtin_amdgcn_exp2f(y);
      r.s += e;
      r.t += e * fmaxf(y, -1000.f);  // e = 0 there
    }
    if (TOP && __ballot(valid && list.wants(vm))) {
#pragma unroll
      for (int j = 0; j < c; ++j)
        list.insert(valid ? order_of(f[j]) : 0, valid ? ~(uint32_t)(id0 + j) : 0, top, lane);
    }
  };
  using One = std::integral_constant<int, 1>;
  using Vec = std::integral_constant<int, E>;

  // the part's logits up to the first 16-byte border, and past the last
  const int64_t off = (int64_t)(((uintptr_t)(row + lo) & 15u) / sizeof(T));
  int64_t head = off ? E - off : 0;
  if (head > hi - lo) head = hi - lo;
  const int64_t nv = (hi - lo - head) / E, tail0 = lo + head + nv * E;
  if (w == 0 && (head > 0 || tail0 < hi)) {
    const bool is_head = lane < head, is_tail = lane >= 32 && tail0 + lane - 32 < hi;
    const int64_t id = is_head ? lo + lane : tail0 + lane - 32;
    float f[1] = {-INFINITY};
    if (is_head || is_tail) f[0] = Elem<T>::load(row + id);
    take(f, One{}, id, is_head || is_tail);
  }
  const u32x4_t* body = (const u32x4_t*)(row + lo + head);
  for (int64_t v0 = 0; v0 < nv; v0 += (int64_t)kLpThreads * U) {
    u32x4_t raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + u * kLpThreads + tid;
      if (v < nv) raw[u] = body[v];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + u * kLpThreads + tid;
      if (v0 + u * kLpThreads + w * 64 >= nv) break;  // no lane of the wave
      float f[E];
      if (v < nv) {
        unpack<T>(raw[u], f);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = -INFINITY;
      }
      take(f, Vec{}, lo + head + v * E, v < nv);
    }
  }
  // the waves' sums on one reference, their lists as one
  r.s = wave_sum(r.s);
  r.t = wave_sum(r.t);
  if (lane == 0) sums[w] = r;
  if (TOP) {
    if (lane < top) keys[w * top + lane] = ((uint64_t)list.hi << 32) | list.lo;
    if (tid < top) best[tid] = 0;
  }
  __syncthreads();
  RowSums a = sums[0];
#pragma unroll
  for (int k = 1; k < kLpWaves; ++k) {
    RowSums b = sums[k];
    const float to = fmaxf(a.m, b.m);
    a.move(to, c2);
    b.move(to, c2);
    a.s += b.s;
    a.t += b.t;
  }
  if (TOP) {
    if (tid < kLpWaves * top) {
      const uint64_t k = keys[tid];
      int rank = 0;
      for (int i = 0; i < kLpWaves * top; ++i) rank += keys[i] > k;
      if (k != 0 && rank < top) best[rank] = k;
    }
    __syncthreads();
  }
  if (parts == 1) {
    finish_row<T>(out, n, row, targets, V, scale, TOP ? top : 0, a, best, tid);
  } else {
    if (tid == 0) wsum[blockIdx.x] = f32x4_t{a.m, a.s, a.t, 0.f};
    if (TOP && tid < top) wkey[(int64_t)blockIdx.x * top + tid] = best[tid];
  }
}

// A wave per row: lane i holds part i's sums and, of its list, the largest
// key not yet taken.
template <typename T>
__global__ void __launch_bounds__(64) logprob_join_kernel(const T* logits, const void* targets, int64_t V, int64_t ld,
                                                          float scale, int top, int parts, LogprobOut out,
                                                          const uint64_t* wkey, const f32x4_t* wsum) {
  __shared__ uint64_t best[LSTM_MAX_TOP];
  const int lane = threadIdx.x;
  const int64_t n = blockIdx.x;
  const float c2 = scale * kLog2e;
  RowSums r = {-INFINITY, 0.f, 0.f};
  if (lane < parts) {
    const f32x4_t q = wsum[n * parts + lane];
    r = RowSums{q[0], q[1], q[2]};
  }
  r.move(wave_max(r.m), c2);
  r.s = wave_sum(r.s);
  r.t = wave_sum(r.t);
  const uint64_t* mine = wkey + (n * parts + lane) * top;
  int at = 0;
  uint64_t head = lane < parts && top > 0 ? mine[0] : 0;
  for (int k = 0; k < top; ++k) {
    uint64_t big = head;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor((unsigned long long)big, o);
      big = other > big ? other : big;
    }
    if (lane == 0) best[k] = big;
    if (head == big && big != 0) {
      ++at;
      head = at < top ? mine[at] : 0;
    }
  }
  __syncthreads();
  finish_row<T>(out, n, logits + n * ld, targets, V, scale, top, r, best, lane);
}

// ---------------------------------------------------------------------------
// Gradient: a work-group per (row, chunk of kGradVecs vectors a thread); the
// few elements that have a term of their own (the target, the alternatives)
// are written again by the group that owns them.
constexpr int kGradVecs = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kLpThreads) logprob_bwd_kernel(const T* logits, const void* targets,
                                                                 const float* record, const float* entropy, const void* top_ids,
                                                                 const float* dlogp, const float* dentropy,
                                                                 const float* dtop, T* dlogits, int64_t V, int64_t ld,
                                                                 int64_t ldg, float scale, int top, int id64,
                                                                 int chunks) {
  constexpr int E = VEC ? vec_of<T>() : 1;
  constexpr int U = VEC ? kGradVecs : kGradVecs * vec_of<T>();
  constexpr int64_t kSpan = (int64_t)kLpThreads * U;
  const int tid = threadIdx.x;
  const int64_t n = blockIdx.x / chunks, ch = blockIdx.x - n * chunks;
  const T* row = logits + n * ld;
  T* grad = dlogits + n * ldg;
  const float m = record[2 * n], ls = record[2 * n + 1];
  const bool none = m == -INFINITY;
  const float H = dentropy ? entropy[n] : 0.f, gH = dentropy ? dentropy[n] : 0.f;
  int64_t target = -1;
  float gl = 0.f;
  if (dlogp) {
    target = id_at(targets, n, id64);
    if (target < 0 || target >= V) target = -1;
    else gl = dlogp[n];
  }
  float G = gl;
  if (dtop)
    for (int k = 0; k < top; ++k) G += dtop[n * top + k];
  // scale (-p (G + gH (log p + H)));  p = 0: 0, log p kept finite.  The
  // exponential gives 0 below 2^-126: p is carried 2^32 times larger up to
  // the last product.
  const float out_scale = -scale * 2.3283064365386963e-10f;
  auto value = [&](float x) {
    const float lp = (x - m) * scale - ls, p = __builtin_amdgcn_exp2f(__builtin_fmaf(lp, kLog2e, 32.f));
    return none ? 0.f : out_scale * (p * (G + gH * (fmaxf(lp, -1000.f) + H)));
  };
  const int64_t off = VEC ? (int64_t)(((uintptr_t)row & 15u) / sizeof(T)) : 0;
  int64_t head = off ? E - off : 0;
  if (head > V) head = V;
  const int64_t nv = (V - head) / E, tail0 = head + nv * E;
  const int64_t v0 = ch * kSpan;
  // the own elements this group writes: thread 0 the target, 1 .. top the
  // alternatives (the first of equal ids), read before anything is written
  int64_t own = -1;
  float own_g = 0.f;
  if (tid <= top) {
    own = tid == 0 ? target : dtop ? id_at(top_ids, n * top + tid - 1, id64) : -1;
    if (tid > 0 && own == target) own = -1;
    if (own >= V) own = -1;
    if (own >= 0) {
      const bool edge = own < head || own >= tail0;
      const int64_t of = edge ? 0 : (own - head) / E / kSpan;
      if (of != ch) own = -1;
    }
    if (own >= 0) {
      float g = own == target ? gl : 0.f;
      if (dtop)
        for (int k = 0; k < top; ++k) g += id_at(top_ids, n * top + k, id64) == own ? dtop[n * top + k] : 0.f;
      own_g = none ? 0.f : value(Elem<T>::load(row + own)) + scale * g;
    }
  }
  __syncthreads();
  if (ch == 0 && (tid < head || (tid >= 64 && tail0 + tid - 64 < V))) {
    const int64_t i = tid < head ? tid : tail0 + tid - 64;
    grad[i] = Elem<T>::from_f(as_f32(value(Elem<T>::load(row + i))));
  }
  if constexpr (VEC) {
    const u32x4_t* src = (const u32x4_t*)(row + head);
    u32x4_t* dst = (u32x4_t*)(grad + head);
    u32x4_t raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + u * kLpThreads + tid;
      if (v < nv) raw[u] = src[v];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + u * kLpThreads + tid;
      if (v < nv) {
        float f[E];
        unpack<T>(raw[u], f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = value(f[j]);
        dst[v] = pack<T>(f);
      }
    }
  } else {
#pragma unroll 4
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + u * kLpThreads + tid;
      if (v < nv) grad[v] = Elem<T>::from_f(as_f32(value(Elem<T>::load(row + v))));
    }
  }
  __syncthreads();  // the group's stores are done in its order
  if (own >= 0) grad[own] = Elem<T>::from_f(own_g);
}

// ---------------------------------------------------------------------------
template <typename T>
static hipError_t logprob_fwd_t(const LogprobPlan& p, const void* logits, const void* targets, char* ws,
                                const LogprobOut& o, hipStream_t s) {
  uint64_t* wkey = (uint64_t*)(ws + p.off_key);
  f32x4_t* wsum = (f32x4_t*)(ws + p.off_sum);
  const unsigned grid = (unsigned)(p.N * p.parts);
  if (p.top > 0)
    logprob_fwd_kernel<T, true><<<grid, kLpThreads, 0, s>>>((const T*)logits, targets, p.V, p.ld, p.scale, p.top,
                                                            p.parts, p.part, o, wkey, wsum);
  else
    logprob_fwd_kernel<T, false><<<grid, kLpThreads, 0, s>>>((const T*)logits, targets, p.V, p.ld, p.scale, 0, p.parts,
                                                             p.part, o, wkey, wsum);
  if (p.parts > 1)
    logprob_join_kernel<T><<<(unsigned)p.N, 64, 0, s>>>((const T*)logits, targets, p.V, p.ld, p.scale, p.top, p.parts,
                                                        o, wkey, wsum);
  return hipGetLastError();
}

hipError_t launch_logprob_fwd(const LogprobPlan& p, const void* logits, const void* targets, char* ws, float* record,
                              float* lse, float* logp, float* entropy, float* top_logp, void* top_ids, hipStream_t s) {
  if (p.N == 0) return hipSuccess;
  Timed tm(9, s);
  const LogprobOut o = {record, lse, logp, entropy, top_logp, top_ids, p.id64};
  if (p.dtype == LSTM_F32) return logprob_fwd_t<float>(p, logits, targets, ws, o, s);
  if (p.dtype == LSTM_BF16) return logprob_fwd_t<bf16_t>(p, logits, targets, ws, o, s);
  return logprob_fwd_t<f16_t>(p, logits, targets, ws, o, s);
}

template <typename T>
static hipError_t logprob_bwd_t(const LogprobPlan& p, const void* logits, const void* targets, const float* record,
                                const float* entropy, const void* top_ids, const float* dlogp, const float* dentropy,
                                const float* dtop, void* dlogits, hipStream_t s) {
  // rows of logits and dlogits that lie alike against 16 bytes
  const bool v = ((uintptr_t)logits & 15u) == ((uintptr_t)dlogits & 15u) &&
                 ((p.ld - p.ldg) * (int64_t)sizeof(T)) % 16 == 0;
  const int64_t span = (int64_t)kLpThreads * kGradVecs * vec_of<T>();
  const int chunks = (int)((p.V + span - 1) / span);
  const unsigned grid = (unsigned)(p.N * chunks);
  const int top = dtop ? p.top : 0;
  if (v)
    logprob_bwd_kernel<T, true><<<grid, kLpThreads, 0, s>>>((const T*)logits, targets, record, entropy, top_ids, dlogp,
                                                            dentropy, dtop, (T*)dlogits, p.V, p.ld, p.ldg, p.scale, top,
                                                            p.id64, chunks);
  else
    logprob_bwd_kernel<T, false><<<grid, kLpThreads, 0, s>>>((const T*)logits, targets, record, entropy, top_ids, dlogp,
                                                             dentropy, dtop, (T*)dlogits, p.V, p.ld, p.ldg, p.scale,
                                                             top, p.id64, chunks);
  return hipGetLastError();
}

hipError_t launch_logprob_bwd(const LogprobPlan& p, const void* logits, const void* targets, const float* record,
                              const float* entropy, const void* top_ids, const float* dlogp, const float* dentropy,
                              const float* dtop, void* dlogits, hipStream_t s) {
  if (p.N == 0 || p.V == 0) return hipSuccess;
  Timed tm(9, s);
  if (p.dtype == LSTM_F32)
    return logprob_bwd_t<float>(p, logits, targets, record, entropy, top_ids, dlogp, dentropy, dtop, dlogits, s);
  if (p.dtype == LSTM_BF16)
    return logprob_bwd_t<bf16_t>(p, logits, targets, record, entropy, top_ids, dlogp, dentropy, dtop, dlogits, s);
  return logprob_bwd_t<f16_t>(p, logits, targets, record, entropy, top_ids, dlogp, dentropy, dtop, dlogits, s);
}

}  // namespace lstm
