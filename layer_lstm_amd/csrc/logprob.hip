// logprob.hip -- log probabilities of given tokens, entropy, best
// alternatives, and the logits' gradient (gfx950).
//
// One pass over a row keeps, against the largest logit m of the wave so far,
// the number c of logits equal to m and, per lane, s = sum 2^y and t = sum 2^y y
// of y = (x - m) scale log2(e) over the others, so that
//   log sum exp(scale (x - m)) = log1p(c - 1 + s) =: ls,
//   lse = scale m + ls,   entropy = ls - ln 2 t / (c + s),
//   log p = scale (x - m) - ls,
// the last without the rounding of lse, which for logits of large magnitude
// (a row of the type's lowest value, say) would be all of the result: the
// gradient therefore reads m and ls (the record) and not lse.  The largest
// logits' own 1 stays out of the sum so that where one token has nearly all of
// p, ls and with it 1 - p keep all their digits: in s = 1 + 10^-5 they would be
// two.  A new m, of which a row has few, rescales the sums.
//
// The alternatives are kept as a list sorted across the lanes of a wave: a
// 64-bit key per lane, the logit in an order-preserving form above the
// complement of its id, so that no two keys are equal and a tie goes to the
// lower id.  Logits that reach the list's entry `top` are appended to a buffer
// in LDS, and a full buffer is merged into the list by counting, for every
// key, the keys above it.
#include <type_traits>

#include "internal.hpp"
#include "seq_internal.hpp"

namespace lstm {

constexpr int kLpThreads = 256;
constexpr int kLpVecs = 4;      // 16-byte vectors a lane of the forward takes at a time
constexpr int kMaxParts = 64;   // a row's parts are joined by the lanes of one wave

void make_logprob_plan(const lstm_logprob_shape& s, int cus, LogprobPlan* p) {
  p->N = s.N; p->V = s.V; p->ld = s.ld; p->ldg = s.ld_grad;
  p->scale = s.scale; p->top = s.top; p->dtype = s.dtype; p->id64 = s.id_type == LSTM_I64;
  // a wave per row; rows too few for eight waves a compute unit are split,
  // down to one round of a wave's loads
  const int64_t step = (int64_t)64 * kLpVecs * (s.dtype == LSTM_F32 ? 4 : 8);
  int64_t parts = 1;
  if (s.N > 0 && s.N < 8 * (int64_t)cus) parts = 8 * (int64_t)cus / s.N;
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

// A logit as an unsigned integer of the same order (-0 taken as +0; NaN of
// either sign above all others, so that it has a place in the list).
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return x != x ? 0xffffffffu : u ^ (uint32_t)(((int32_t)u >> 31) | (int32_t)0x80000000);
}
__device__ __forceinline__ float from_order(uint32_t o) {
  return __uint_as_float(o ^ ((o & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// Reductions over a wave in registers: inside rows of 16 lanes by row_shr,
// then across the rows by row_bcast, the result in lane 63 (in a fixed order).
template <class Op>
__device__ __forceinline__ float wave_reduce(float v, float none, Op op) {
  auto from = [&](auto ctl, auto rows) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        (int)__float_as_uint(none), (int)__float_as_uint(v), decltype(ctl)::value, decltype(rows)::value, 0xf, false));
  };
  using std::integral_constant;
  v = op(v, from(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{}));  // row_shr:1
  v = op(v, from(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{}));  // row_shr:2
  v = op(v, from(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{}));  // row_shr:4
  v = op(v, from(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{}));  // row_shr:8
  v = op(v, from(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{}));  // row_bcast:15 into rows 1, 3
  v = op(v, from(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{}));  // row_bcast:31 into rows 2, 3
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_reduce(v, 0.f, [](float a, float b) { return a + b; });
}

// Sums against a reference m, the largest logit seen: s = sum 2^y, t = sum 2^y
// y over smaller ones, c the number of those equal to it.  y is one fused
// multiply-add, x c2 - m2 with m2 = m c2 rounded; the rounding of m2, which is
// the y of m itself, is taken off when the sums are read (lost).  Where m c2
// might overflow (a row of the type's lowest value) y = (x - m) c2 and m2 = 0.
struct RowSums {
  float m, s, t, c;  // m = -inf: nothing but -inf so far (s = t = c = 0, or NaN)
  __device__ __forceinline__ bool huge(float c2) const { return !(fabsf(m * c2) < 1e37f); }
  __device__ __forceinline__ float m2(float c2) const { return huge(c2) ? 0.f : m * c2; }
  __device__ __forceinline__ float lost(float c2) const { return huge(c2) ? 0.f : __builtin_fmaf(m, c2, -m2(c2)); }
  __device__ __forceinline__ void move(float to, float c2) {
    if (m != -INFINITY && to != m) {
      RowSums n = {to, 0.f, 0.f, 0.f};
      const float d = !huge(c2) && !n.huge(c2) ? n.m2(c2) - m2(c2) : (to - m) * c2;
      const float r = __builtin_amdgcn_exp2f(-d), y = lost(c2), own = c * __builtin_amdgcn_exp2f(y), all = s + own;
      t = r == 0.f ? all * 0.f : (__builtin_fmaf(own, y, t) - d * all) * r;
      s = all * r;
      c = 0.f;
    }
    m = to;
  }
  // log sum exp(scale (x - m)), and the entropy
  __device__ __forceinline__ void read(float c2, float* ls, float* entropy) const {
    const float y = lost(c2), k = __builtin_amdgcn_exp2f(-y), rest = (c - 1.f) + s * k;
    *ls = log1pf(rest);
    *entropy = m == -INFINITY && s == 0.f ? 0.f : *ls - kLn2 * (k * __builtin_fmaf(-y, s, t)) / (1.f + rest);
  }
};

// The largest threshold that at least `top` of the wave's values reach, on the
// grid of the upper kGridBits bits (0: fewer than `top` values).  Values are
// order_of() of one logit per lane, 0 for none.
constexpr int kGridBits = 16;
__device__ __forceinline__ uint32_t wave_threshold(uint32_t v, int top) {
  uint32_t at = 0;
#pragma unroll
  for (int b = 31; b >= 32 - kGridBits; --b) {
    const uint32_t to = at | (1u << b);
    if (__popcll(__ballot(v >= to)) >= top) at = to;
  }
  return at;
}

// The value of f whose bit alone is set (registers cannot be indexed).
template <int C>
__device__ __forceinline__ float pick(const float* f, uint32_t bit) {
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) v |= __float_as_uint(f[i]) & (uint32_t)__builtin_amdgcn_sbfe((int)bit, i, 1);
  return __uint_as_float(v);
}

// What a wave's list needs in LDS: the keys appended since the last merge,
// and the merged keys in order.
struct TopLds {
  uint64_t cand[128], sorted[LSTM_MAX_TOP];
};
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The list: lane i < top holds the i-th largest key so far (0: none).  A key
// has to pass `least`: the list's last, or a floor that `top` logits of the
// wave are known to reach (which keeps the first logits of a row from being
// appended one and all).
struct TopList {
  uint64_t key, least;
  float tval;  // the logit of `least` (no number where everything may pass)
  int count;   // appended keys
  __device__ __forceinline__ void clear() { key = least = 0; tval = -NAN; count = 0; }
  __device__ __forceinline__ void set_floor(uint32_t order) {
    if (order > 0) {
      least = ((uint64_t)order << 32) - 1;
      tval = from_order(order);
    }
  }
  // true where x may be a key to append
  __device__ __forceinline__ bool wants(float x) const { return !(x < tval); }
  // one key of every lane (0: none), and a merge as soon as it can raise the
  // list's last key; `more`: further keys follow at once
  __device__ __forceinline__ void append(TopLds* lds, uint64_t k, bool more, int top, int lane) {
    const uint64_t in = __ballot(k > least);
    if (k > least) lds->cand[count + __popcll(in & (((uint64_t)1 << lane) - 1))] = k;
    count += __popcll(in);
    if (count > 64 || (!more && count >= top)) merge(lds, top, lane);
  }
  // appended keys into the list, 64 - top at a time
  __device__ __forceinline__ void merge(TopLds* lds, int top, int lane) {
    wave_sync();
    while (count > 0) {
      const int m = count < 64 - top ? count : 64 - top;
      count -= m;
      uint64_t k = lane < top ? key : 0;
      if (lane >= top && lane < top + m) k = lds->cand[count + lane - top];
      int rank = 0;
      for (int i = 0; i < top + m; i += 4) {
#pragma unroll
        for (int j = i; j < i + 4; ++j) {  // lanes past the last hold no key
          const uint64_t o = ((uint64_t)__builtin_amdgcn_readlane((uint32_t)(k >> 32), j) << 32) |
                             (uint32_t)__builtin_amdgcn_readlane((uint32_t)k, j);
          rank += o > k;
        }
      }
      if (lane < top) lds->sorted[lane] = 0;
      wave_sync();
      if (k != 0 && rank < top) lds->sorted[rank] = k;
      wave_sync();
      key = lane < top ? lds->sorted[lane] : 0;
      const uint64_t last = ((uint64_t)__builtin_amdgcn_readlane((uint32_t)(key >> 32), top - 1) << 32) |
                            (uint32_t)__builtin_amdgcn_readlane((uint32_t)key, top - 1);
      if (last > least) {
        least = last;
        tval = from_order((uint32_t)(last >> 32));
      }
    }
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

// (m, ls): a row's record.  Without a number above -inf m is -inf, and ls -inf,
// or NaN where the row has one.
__device__ __forceinline__ float log_prob(float x, float scale, float m, float ls) {
  return m == -INFINITY ? ls : (x - m) * scale - ls;
}

// The target's logit, which lane 32 of the wave that writes a row reads
// ahead (`real`: the row has one).
struct Target {
  float x;
  bool real;
};
template <typename T>
__device__ __forceinline__ Target read_target(const LogprobOut& o, int64_t n, const T* row, const void* targets,
                                              int64_t V, int tid) {
  Target t = {0.f, false};
  if (tid == 32 && o.logp) {
    const int64_t id = id_at(targets, n, o.id64);
    t.real = id >= 0 && id < V;
    if (t.real) t.x = Elem<T>::load(row + id);
  }
  return t;
}

// A row's results from its sums, by one wave; lane i holds key i of the list.
__device__ __forceinline__ void finish_row(const LogprobOut& o, int64_t n, Target target, float scale, int top,
                                           RowSums r, uint64_t key, int tid) {
  float ls, entropy;
  r.read(scale * kLog2e, &ls, &entropy);
  if (tid == 0) {
    o.record[2 * n] = r.m;
    o.record[2 * n + 1] = ls;
    if (o.lse) o.lse[n] = r.m * scale + ls;
    if (o.entropy) o.entropy[n] = entropy;
  }
  if (tid == 32 && o.logp) o.logp[n] = target.real ? log_prob(target.x, scale, r.m, ls) : 0.f;
  if (tid < top) {
    const uint32_t id = ~(uint32_t)key;
    o.top_logp[n * top + tid] = log_prob(from_order((uint32_t)(key >> 32)), scale, r.m, ls);
    if (o.id64) ((int64_t*)o.top_ids)[n * top + tid] = id;
    else ((int32_t*)o.top_ids)[n * top + tid] = (int32_t)id;
  }
}

// A wave per (row, part): the fixed work (joins of sums and lists, threshold)
// is paid once per wave and covered by the row's hundred and more logits per
// lane.  (2049 rows of 10007 fp16 logits with 5 alternatives: 20 us, where a
// work-group of four waves per row and its joins in LDS took a third more; 16
// rows of 131072 fp32 with 8, in 64 parts a row: 7 us and 4 for the join, with
// work-groups 11 and 4.)  A logit costs nine vector instructions with the
// exponential: 16384 rows of 32768 bf16 take 200-235 us, 4.6-5.4 TB/s, the
// vector units 65 % busy.  On the 2049 rows of 10007 the fixed work and the
// list double the instructions, two waves a SIMD do not cover the wait for the
// loads, and neither memory nor the vector units (41 %) are the bound.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kLpThreads) logprob_fwd_kernel(const T* logits, const void* targets, int64_t N,
                                                                 int64_t V, int64_t ld, float scale, int top, int parts,
                                                                 int64_t part, LogprobOut out, uint64_t* wkey,
                                                                 f32x4_t* wsum) {
  constexpr int E = vec_of<T>();
  constexpr int U = kLpVecs;
  __shared__ TopLds tops[TOP ? 4 : 1];
  TopLds* lds = tops + (TOP ? threadIdx.x >> 6 : 0);
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n = parts == 1 ? unit : unit / parts;
  if (n >= N) return;
  const int pt = (int)(unit - n * parts);
  const T* row = logits + n * ld;
  const int64_t lo = (int64_t)pt * part, hi = lo + part < V ? lo + part : V;
  const float c2 = scale * kLog2e;
  Target target = {0.f, false};
  if (parts == 1) target = read_target<T>(out, n, row, targets, V, lane);

  RowSums r = {-INFINITY, 0.f, 0.f, 0.f};
  TopList list;
  list.clear();
  const uint32_t count = (uint32_t)(hi - lo);
  // C logits of this lane, E at a time 64 E apart, the first at id0 of the
  // part; from id `end` on -inf stands for them and they are nobody's keys
  auto take = [&](float* f, auto C, uint32_t id0, uint32_t end) {
    constexpr int c = decltype(C)::value;
    // maxima of groups of up to eight and of all, NaN if one of them is (for the list)
    constexpr int kPer = c < 8 ? c : 8;
    float gm[c / kPer], vm = -INFINITY;
#pragma unroll
    for (int g = 0; g < c / kPer; ++g) {
      gm[g] = f[g * kPer];
#pragma unroll
      for (int j = 1; j < kPer; ++j) gm[g] = __builtin_elementwise_maximum(gm[g], f[g * kPer + j]);
      vm = __builtin_elementwise_maximum(vm, gm[g]);
    }
    if (__ballot(vm > r.m)) r.move(fmaxf(wave_max(vm), r.m), c2);
    if (TOP && __ballot(list.wants(vm))) {
      // each lane's candidates as bits, then one of every lane at a time
      // (mostly there is one in all)
      uint32_t bits = 0;
#pragma unroll
      for (int j = 0; j < c; ++j) bits |= list.wants(f[j]) ? 1u << j : 0u;
      while (__ballot(bits != 0)) {
        const int j = bits ? __builtin_ctz(bits) : 0;
        const uint32_t id = id0 + (j / E) * (64 * E) + j % E;
        const bool in = bits != 0 && id < end;
        const uint64_t key = ((uint64_t)order_of(pick<c>(f, bits & -bits)) << 32) | ~((uint32_t)lo + id);
        bits &= bits - 1;
        list.append(lds, in ? key : 0, __ballot(bits != 0) != 0, top, lane);
      }
    }
    if (__ballot(vm == r.m && fabsf(vm) < INFINITY)) {  // counted, not summed
#pragma unroll
      for (int g = 0; g < c / kPer; ++g) {
        if (!__ballot(gm[g] == r.m)) continue;
#pragma unroll
        for (int j = g * kPer; j < (g + 1) * kPer; ++j) {
          const bool is = f[j] == r.m;
          r.c += is ? 1.f : 0.f;
          f[j] = is ? -INFINITY : f[j];
        }
      }
    }
    const bool huge = r.huge(c2) && r.m != -INFINITY;
    if (huge) {
#pragma unroll
      for (int j = 0; j < c; ++j) f[j] -= r.m;
    }
    const float m2 = huge || r.m == -INFINITY ? 0.f : r.m * c2;
#pragma unroll
    for (int j = 0; j < c; ++j) {
      const float y = __builtin_fmaf(f[j], c2, -m2), e = __builtin_amdgcn_exp2f(y);
      r.s += e;
      r.t += e * fmaxf(y, -1000.f);  // e = 0 there
    }
  };
  using One = std::integral_constant<int, 1>;
  using Take = std::integral_constant<int, U * E>;

  // the part's logits up to the first 16-byte border, and past the last
  const uint32_t off = (uint32_t)(((uintptr_t)(row + lo) & 15u) / sizeof(T));
  uint32_t head = off ? E - off : 0;
  if (head > count) head = count;
  const uint32_t nv = (count - head) / E, tail0 = head + nv * E;
  const u32x4_t* body = (const u32x4_t*)(row + lo + head);
  u32x4_t raw[U], none;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    none[j] = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, f16_t>::value ? 0xfc00fc00u : 0xff80ff80u;  // -inf
  auto fetch = [&](uint32_t v0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t v = v0 + u * 64 + lane;
      raw[u] = none;
      if (v < nv) raw[u] = body[v];
    }
  };
  fetch(0);
  const bool is_head = lane < (int)head, is_tail = lane >= 32 && tail0 + lane - 32 < count;
  float edge[1] = {-INFINITY};
  const uint32_t edge_id = is_head ? lane : is_tail ? tail0 + lane - 32 : count;
  if (is_head || is_tail) edge[0] = Elem<T>::load(row + lo + edge_id);
  if (TOP) {
    float vm = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[E];
      unpack<T>(raw[u], f);
#pragma unroll
      for (int j = 0; j < E; ++j) vm = fmaxf(vm, f[j]);
    }
    list.set_floor(wave_threshold(lane < (int)nv ? order_of(vm) : 0, top));
  }
  if (head > 0 || tail0 < count) take(edge, One{}, edge_id, count);
#pragma unroll 1
  for (uint32_t v0 = 0; v0 < nv; v0 += 64 * U) {  // one copy of its long body: the next loads run beside it
    float f[U * E];
#pragma unroll
    for (int u = 0; u < U; ++u) unpack<T>(raw[u], f + u * E);
    if (v0 + 64 * U < nv) fetch(v0 + 64 * U);
    take(f, Take{}, head + (v0 + lane) * E, tail0);
  }
  if (TOP) list.merge(lds, top, lane);
  r.s = wave_sum(r.s);
  r.t = wave_sum(r.t);
  r.c = wave_sum(r.c);
  if (parts == 1) {
    finish_row(out, n, target, scale, TOP ? top : 0, r, list.key, lane);
  } else {
    if (lane == 0) wsum[unit] = f32x4_t{r.m, r.s, r.t, r.c};
    if (TOP && lane < top) wkey[unit * top + lane] = list.key;
  }
}

// A wave per row: lane i holds part i's sums and, of its list, the largest
// key not yet taken.
template <typename T>
__global__ void __launch_bounds__(64) logprob_join_kernel(const T* logits, const void* targets, int64_t V, int64_t ld,
                                                          float scale, int top, int parts, LogprobOut out,
                                                          const uint64_t* wkey, const f32x4_t* wsum) {
  const int lane = threadIdx.x;
  const int64_t n = blockIdx.x;
  const float c2 = scale * kLog2e;
  const Target target = read_target<T>(out, n, logits + n * ld, targets, V, lane);
  RowSums r = {-INFINITY, 0.f, 0.f, 0.f};
  if (lane < parts) {
    const f32x4_t q = wsum[n * parts + lane];
    r = RowSums{q[0], q[1], q[2], q[3]};
  }
  r.move(wave_max(r.m), c2);
  r.s = wave_sum(r.s);
  r.t = wave_sum(r.t);
  r.c = wave_sum(r.c);
  __shared__ TopLds lds;
  TopList list;
  list.clear();
  if (top > 0) {
    // the lists' largest keys bound the key `top` of all from below
    const uint64_t* mine = wkey + (n * parts + lane) * top;
    uint64_t key = lane < parts ? mine[0] : 0;
    list.set_floor(wave_threshold((uint32_t)(key >> 32), top));
    for (int k = 0; k < top; ++k) {
      if (!__ballot(key > list.least)) break;  // the lists descend
      const uint64_t now = key;
      key = k + 1 < top && lane < parts ? mine[k + 1] : 0;
      list.append(&lds, now, k + 1 < top, top, lane);
    }
    list.merge(&lds, top, lane);
  }
  finish_row(out, n, target, scale, top, r, list.key, lane);
}

// ---------------------------------------------------------------------------
// Gradient: a work-group per (row, chunk of kGradVecs vectors a thread); the
// few elements that have a term of their own (the target, the alternatives)
// are written again by the group that owns them.  One read and one write of
// the logits are all it moves: 16384 x 32768 bf16, 2.15 GB, 355-380 us, 5.9
// TB/s, with the vector units 84 % busy beside the memory.
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
  const bool none = m == -INFINITY && ls == -INFINITY;
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
  // the last product, as the square of 2^16 sqrt(p).  (The factor in the
  // exponent, y + 32, would round a p near 1 to 2^-19 of itself; one that raises
  // small exponents alone takes 16384 x 32768 bf16 396 us.)
  const float out_scale = -scale * 2.3283064365386963e-10f;
  auto log_p = [&](float x) { return __builtin_fmaf(x - m, scale, -ls); };
  auto value = [&](float x) {
    const float lp = log_p(x), h = __builtin_amdgcn_exp2f(lp * (kLog2e / 2)) * 0x1p16f;
    return none ? 0.f : out_scale * (h * h * (G + gH * (fmaxf(lp, -1000.f) + H)));
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
      float g = own == target ? gl : 0.f, other = own == target ? 0.f : gl;  // its cotangents, the others'
      if (dtop)
        for (int k = 0; k < top; ++k) {
          const float v = dtop[n * top + k];
          const bool mine = id_at(top_ids, n * top + k, id64) == own;
          g += mine ? v : 0.f;
          other += mine ? 0.f : v;
        }
      // g - p G of a p near 1 by 1 - p = -expm1(log p), which keeps its digits
      const float x = Elem<T>::load(row + own), lp = log_p(x), less = expm1f(lp);
      own_g = none        ? 0.f
              : lp > -.5f ? -scale * (other + __builtin_fmaf(G, less, gH * (lp + H) * (1.f + less)))
                          : value(x) + scale * g;
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
  const unsigned grid = (unsigned)((p.N * p.parts + 3) / 4);
  if (p.top > 0)
    logprob_fwd_kernel<T, true><<<grid, kLpThreads, 0, s>>>((const T*)logits, targets, p.N, p.V, p.ld, p.scale,
                                                            p.top, p.parts, p.part, o, wkey, wsum);
  else
    logprob_fwd_kernel<T, false><<<grid, kLpThreads, 0, s>>>((const T*)logits, targets, p.N, p.V, p.ld, p.scale, 0,
                                                             p.parts, p.part, o, wkey, wsum);
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
  const int64_t step = kMaxGroups / chunks;  // rows a launch
  const int top = dtop ? p.top : 0, ids = p.id64 ? 8 : 4;
  for (int64_t n = 0; n < p.N; n += step) {
    const unsigned grid = (unsigned)((p.N - n < step ? p.N - n : step) * chunks);
    auto from = [n](const auto* at, int64_t row) { return at ? at + n * row : nullptr; };
    auto launch = [&](auto vec) {
      logprob_bwd_kernel<T, decltype(vec)::value><<<grid, kLpThreads, 0, s>>>(
          (const T*)logits + n * p.ld, from((const char*)targets, ids), record + 2 * n, from(entropy, 1),
          from((const char*)top_ids, (int64_t)ids * p.top), from(dlogp, 1), from(dentropy, 1), from(dtop, p.top),
          (T*)dlogits + n * p.ldg, p.V, p.ld, p.ldg, p.scale, top, p.id64, chunks);
    };
    if (v) launch(std::true_type{});
    else launch(std::false_type{});
  }
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
