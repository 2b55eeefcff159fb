// embed.hip -- token embedding and the gradient of its table (gfx950).
//
//   out[n] = scale * table[ids[n]]        dtable[v] = scale * sum_{ids[n]=v} dout[n]
//
// The forward is a copy of rows.  The gradient sorts the tokens by id with a
// stable radix sort (so that the sum of a row runs over n in ascending order
// and every call gives the same bits), sums the whole chunks of kChunk sorted
// positions that hold one id alone, and then writes every row of dtable from
// its range of the sorted tokens: the rows of a chunk that it shares with
// other ids one by one, its whole chunks by their sums.  A row therefore
// costs at most 2 kChunk rows of dout and one sum per chunk, whatever its
// share of the tokens.
#include "internal.hpp"
#include "seq_internal.hpp"

namespace lstm {

constexpr int kChunk = 64;         // sorted positions per chunk
constexpr int kMaxDigit = 11;      // bits per pass of the sort
constexpr int kCountSort = 4096;   // up to this many tokens are sorted by counting
constexpr int kEmbThreads = 256;

void make_embed_plan(const lstm_embed_shape& s, EmbedPlan* p) {
  p->N = s.N; p->V = s.V; p->D = s.D;
  p->ldt = s.ld_table; p->ldo = s.ld_out; p->padding = s.padding;
  p->scale = s.scale; p->dtype = s.dtype; p->id64 = s.id_type == LSTM_I64;
  p->bits = 1;  // keys 0 .. V, V standing for tokens without a row
  while (((int64_t)1 << p->bits) <= s.V) ++p->bits;
  p->passes = (p->bits + kMaxDigit - 1) / kMaxDigit;
  p->digit = (p->bits + p->passes - 1) / p->passes;
  // every block of the scatter reads the counts of all blocks: at most 128
  p->rounds = 4;
  while ((s.N + kEmbThreads * (int64_t)p->rounds - 1) / (kEmbThreads * (int64_t)p->rounds) > 128) p->rounds *= 2;
  p->blocks = (int)((s.N + kEmbThreads * (int64_t)p->rounds - 1) / (kEmbThreads * (int64_t)p->rounds));
  size_t off = 0;
  p->off_pair0 = off; off += align256_seq((size_t)s.N * 8);
  p->off_pair1 = off; off += align256_seq((size_t)s.N * 8);
  p->off_hist = off; off += align256_seq(((size_t)p->blocks << p->digit) * 4);
  p->off_seg = off; off += align256_seq((size_t)s.V * 8);
  p->off_part = off; off += align256_seq((size_t)(s.N / kChunk) * (size_t)((s.D + 3) / 4 * 4) * 4);
  p->total = off;
}

// ---------------------------------------------------------------------------
// Rows of D elements, a lane holding E = 16 bytes' worth of each slab of
// 64 E: side by side where every row is 16-byte aligned (VEC), else 64 apart.
template <typename T, bool VEC>
__device__ __forceinline__ void load_slab(const T* row, int64_t col0, int lane, int64_t D, float* f) {
  constexpr int E = vec_of<T>();
  if constexpr (VEC) {
    const int64_t c = col0 + lane * E;
    u32x4_t v = {0, 0, 0, 0};
    if (c < D) v = *(const u32x4_t*)(row + c);
    unpack<T>(v, f);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int64_t c = col0 + lane + 64 * j;
      f[j] = c < D ? Elem<T>::load(row + c) : 0.f;
    }
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_slab(T* row, int64_t col0, int lane, int64_t D, const float* f) {
  constexpr int E = vec_of<T>();
  if constexpr (VEC) {
    const int64_t c = col0 + lane * E;
    if (c < D) *(u32x4_t*)(row + c) = pack<T>(f);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int64_t c = col0 + lane + 64 * j;
      if (c < D) row[c] = Elem<T>::from_f(as_f32(f[j]));
    }
  }
}

// ---------------------------------------------------------------------------
// Forward: a wave per (row, slab).
template <typename T, typename ID, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) embed_fwd_kernel(const ID* ids, const T* table, T* out, int64_t N,
                                                                int64_t V, int64_t D, int64_t ldt, int64_t ldo,
                                                                float scale) {
  constexpr int E = vec_of<T>();
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * 4 + w;
  if (n >= N) return;
  const int64_t id = (int64_t)ids[n];
  const int64_t c = (int64_t)blockIdx.y * 64 * E;
  float f[E];
#pragma unroll
  for (int j = 0; j < E; ++j) f[j] = 0.f;
  if (id >= 0 && id < V) load_slab<T, VEC>(table + id * ldt, c, lane, D, f);
#pragma unroll
  for (int j = 0; j < E; ++j) f[j] *= scale;
  store_slab<T, VEC>(out + n * ldo, c, lane, D, f);
}

// ---------------------------------------------------------------------------
// The sort.  Key of a token: its id, or V where it has no gradient.
template <typename ID>
__device__ __forceinline__ uint32_t key_of(const ID* ids, int64_t n, int64_t V, int64_t padding) {
  const int64_t id = (int64_t)ids[n];
  return (uint32_t)(id >= 0 && id < V && id != padding ? id : V);
}

// The rows' ranges start empty.
__device__ __forceinline__ void clear_segs(uint2* seg, int64_t V) {
  const int64_t n = (int64_t)gridDim.x * blockDim.x;
  for (int64_t v = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; v < V; v += n) seg[v] = make_uint2(0, 0);
}

// Few tokens: the place of a token is the number of tokens before it in
// (key, position) order, counted against all of them in LDS.  A work-group of
// 16 waves places 64 tokens, each wave counting over a sixteenth.
template <typename ID>
__global__ void __launch_bounds__(1024) embed_count_sort(const ID* ids, uint2* out, uint2* seg, int N, int64_t V,
                                                         int64_t padding) {
  __shared__ __attribute__((aligned(16))) uint32_t key[kCountSort];
  __shared__ int part[16][64];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  clear_segs(seg, V);
  const int padded = (N + 63) & ~63;
  for (int i = tid; i < padded; i += 1024) key[i] = i < N ? key_of(ids, i, V, padding) : 0xffffffffu;
  __syncthreads();
  const int i = blockIdx.x * 64 + lane;  // < padded
  const uint32_t mine = key[i];
  int before = 0;
  for (int j = w * 4; j < padded; j += 64) {
    const uint4 k = *(const uint4*)(key + j);
    before += (k.x < mine || (k.x == mine && j < i)) + (k.y < mine || (k.y == mine && j + 1 < i)) +
              (k.z < mine || (k.z == mine && j + 2 < i)) + (k.w < mine || (k.w == mine && j + 3 < i));
  }
  part[w][lane] = before;
  __syncthreads();
  if (w == 0 && i < N) {
    int at = 0;
    for (int k = 0; k < 16; ++k) at += part[k][lane];
    out[at] = make_uint2(mine, (uint32_t)i);
  }
}

// Digit counts of each block's tokens.
template <typename ID, bool FIRST>
__global__ void __launch_bounds__(kEmbThreads) embed_hist(const ID* ids, const uint2* in, uint32_t* hist, uint2* seg,
                                                          int64_t N, int64_t V, int64_t padding, int shift, int digit,
                                                          int rounds) {
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  uint32_t* cnt = (uint32_t*)lds_raw;
  const int bins = 1 << digit, tid = threadIdx.x;
  for (int b = tid; b < bins; b += kEmbThreads) cnt[b] = 0;
  if (FIRST) clear_segs(seg, V);
  __syncthreads();
  const int64_t n0 = (int64_t)blockIdx.x * kEmbThreads * rounds;
  for (int r = 0; r < rounds; ++r) {
    const int64_t n = n0 + r * kEmbThreads + tid;
    if (n < N) {
      const uint32_t k = FIRST ? key_of(ids, n, V, padding) : in[n].x;
      atomicAdd(&cnt[(k >> shift) & (bins - 1)], 1u);
    }
  }
  __syncthreads();
  for (int b = tid; b < bins; b += kEmbThreads) hist[((int64_t)blockIdx.x << digit) + b] = cnt[b];
}

// Stable scatter by one digit: the first place of a digit in a block is the
// number of tokens of lower digits plus that of the digit in the blocks
// before; a wave's tokens follow those of the waves before it, in rounds of
// 64 whose equal digits are found by one ballot per bit.
template <typename ID, bool FIRST>
__global__ void __launch_bounds__(kEmbThreads) embed_scatter(const ID* ids, const uint2* in, uint2* out,
                                                             const uint32_t* hist, int64_t N, int64_t V,
                                                             int64_t padding, int shift, int digit, int rounds) {
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  const int bins = 1 << digit, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  uint32_t* first = (uint32_t*)lds_raw;   // [bins] counts, then first places
  uint32_t* wave = first + bins;          // [4][bins]
  __shared__ uint32_t wsum[4];
  for (int b = tid; b < 4 * bins; b += kEmbThreads) wave[b] = 0;
  // totals of every digit, and this block's offset inside it
  for (int b = tid; b < bins; b += kEmbThreads) {
    uint32_t total = 0, before = 0;
    const uint32_t* h = hist + b;
#pragma unroll 8
    for (int k = 0; k < (int)gridDim.x; ++k) {
      const uint32_t c = h[(int64_t)k << digit];
      if (k < (int)blockIdx.x) before += c;
      total += c;
    }
    first[b] = total;
    wave[b] = before;  // kept in wave 0's row until the totals are summed
  }
  __syncthreads();
  // exclusive sum over the digits, each thread a run of bins / 256 of them
  const int run = bins >= kEmbThreads ? bins / kEmbThreads : 1;
  const bool has = tid * run < bins;
  uint32_t sum = 0;
  if (has)
    for (int b = 0; b < run; ++b) sum += first[tid * run + b];
  uint32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 63) wsum[w] = inc;
  __syncthreads();
  uint32_t at = inc - sum;
  for (int k = 0; k < w; ++k) at += wsum[k];
  if (has)
    for (int b = 0; b < run; ++b) {
      const int i = tid * run + b;
      const uint32_t c = first[i];
      first[i] = at + wave[i];
      at += c;
      wave[i] = 0;
    }
  __syncthreads();
  // the waves' digit counts, then their first places
  const int64_t n0 = (int64_t)blockIdx.x * kEmbThreads * rounds + (int64_t)w * 64 * rounds;
  for (int r = 0; r < rounds; ++r) {
    const int64_t n = n0 + r * 64 + lane;
    if (n < N) {
      const uint32_t k = FIRST ? key_of(ids, n, V, padding) : in[n].x;
      atomicAdd(&wave[w * bins + ((k >> shift) & (bins - 1))], 1u);
    }
  }
  __syncthreads();
  for (int b = tid; b < bins; b += kEmbThreads) {
    uint32_t p = first[b];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t c = wave[k * bins + b];
      wave[k * bins + b] = p;
      p += c;
    }
  }
  __syncthreads();
  volatile uint32_t* place = wave + w * bins;
  for (int r = 0; r < rounds; ++r) {
    const int64_t n = n0 + r * 64 + lane;
    const bool real = n < N;
    uint2 t = make_uint2(0, (uint32_t)n);
    if (real) {
      if (FIRST) t.x = key_of(ids, n, V, padding);
      else t = in[n];
    }
    const uint32_t d = (t.x >> shift) & (bins - 1);
    uint64_t same = __ballot(real);
    for (int b = 0; b < digit; ++b) {
      const uint64_t one = __ballot((d >> b) & 1);
      same &= ((d >> b) & 1) ? one : ~one;
    }
    const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
    const uint32_t p = real ? place[d] : 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (real && rank == 0) place[d] = p + __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (real) out[p + rank] = t;
  }
}

// ---------------------------------------------------------------------------
// Sum of the rows of dout at sorted positions [lo, hi), in order.
template <typename T, bool VEC>
__device__ __forceinline__ void sum_rows(const uint2* sorted, uint32_t lo, uint32_t hi, const T* dout, int64_t ldo,
                                         int64_t c, int lane, int64_t D, float* acc) {
  constexpr int E = vec_of<T>();
  constexpr int U = 4;  // rows in flight
  for (uint32_t p = lo; p < hi; p += 64) {
    const uint32_t m = hi - p < 64 ? hi - p : 64;
    const uint32_t at = (uint32_t)lane < m ? sorted[p + lane].y : 0;
    uint32_t i = 0;
    for (; i + U <= m; i += U) {
      float f[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u)
        load_slab<T, VEC>(dout + (int64_t)(uint32_t)__builtin_amdgcn_readlane(at, i + u) * ldo, c, lane, D, f[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] += f[u][j];
    }
    for (; i < m; ++i) {
      float f[E];
      load_slab<T, VEC>(dout + (int64_t)(uint32_t)__builtin_amdgcn_readlane(at, i) * ldo, c, lane, D, f);
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] += f[j];
    }
  }
}

// A wave per (chunk, slab): the ranges of the ids that start or end in the
// chunk, and the sum of a chunk of one id (partials keep the lanes' order:
// E values side by side).
template <typename T, bool VEC>
__global__ void __launch_bounds__(64) embed_chunks(const uint2* sorted, uint2* seg, float* part, const T* dout,
                                                   int64_t N, int64_t V, int64_t D, int64_t ldo, int64_t ldp) {
  constexpr int E = vec_of<T>();
  const int lane = threadIdx.x;
  const int64_t p0 = (int64_t)blockIdx.x * kChunk, p = p0 + lane;
  const uint32_t key = p < N ? sorted[p].x : (uint32_t)V;
  if (blockIdx.y == 0 && key < (uint32_t)V) {
    if (p == 0 || sorted[p - 1].x != key) seg[key].x = (uint32_t)p;
    if (p + 1 == N || sorted[p + 1].x != key) seg[key].y = (uint32_t)(p + 1);
  }
  const uint32_t k0 = __builtin_amdgcn_readlane(key, 0), k1 = __builtin_amdgcn_readlane(key, 63);
  if (k0 != k1 || k0 == (uint32_t)V) return;
  const int64_t c = (int64_t)blockIdx.y * 64 * E;
  float acc[E];
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = 0.f;
  sum_rows<T, VEC>(sorted, (uint32_t)p0, (uint32_t)(p0 + kChunk), dout, ldo, c, lane, D, acc);
  float* o = part + (int64_t)blockIdx.x * ldp;
  if constexpr (VEC) {
    const int64_t cc = c + lane * E;
    if (cc < D)
#pragma unroll
      for (int j = 0; j < E; j += 4) *(f32x4_t*)(o + cc + j) = f32x4_t{acc[j], acc[j + 1], acc[j + 2], acc[j + 3]};
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (c + lane + 64 * j < D) o[c + lane + 64 * j] = acc[j];
  }
}

// A wave per (row of dtable, slab).  sorted == null: no tokens.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) embed_rows(const uint2* sorted, const uint2* seg, const float* part,
                                                          const T* dout, T* dtable, int64_t V, int64_t D, int64_t ldo,
                                                          int64_t ldt, int64_t ldp, float scale) {
  constexpr int E = vec_of<T>();
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t v = (int64_t)blockIdx.x * 4 + w;
  if (v >= V) return;
  const int64_t c = (int64_t)blockIdx.y * 64 * E;
  float acc[E];
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = 0.f;
  if (sorted) {
    const uint2 sg = seg[v];
    const uint32_t lo = __builtin_amdgcn_readfirstlane(sg.x), hi = __builtin_amdgcn_readfirstlane(sg.y);
    // [lo, a) rows, whole chunks [a, b), [b, hi) rows
    uint32_t a = (lo + kChunk - 1) / kChunk * kChunk, b = hi / kChunk * kChunk;
    if (a > hi) a = hi;
    if (b < a) b = a;
    sum_rows<T, VEC>(sorted, lo, a, dout, ldo, c, lane, D, acc);
#pragma unroll 4
    for (uint32_t k = a / kChunk; k < b / kChunk; ++k) {
      float f[E];
      const float* q = part + (int64_t)k * ldp;
      if constexpr (VEC) {
        const int64_t cc = c + lane * E;
#pragma unroll
        for (int j = 0; j < E; j += 4) {
          f32x4_t x = {0.f, 0.f, 0.f, 0.f};
          if (cc < D) x = *(const f32x4_t*)(q + cc + j);
          f[j] = x[0]; f[j + 1] = x[1]; f[j + 2] = x[2]; f[j + 3] = x[3];
        }
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = c + lane + 64 * j < D ? q[c + lane + 64 * j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] += f[j];
    }
    sum_rows<T, VEC>(sorted, b, hi, dout, ldo, c, lane, D, acc);
  }
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] *= scale;
  store_slab<T, VEC>(dtable + v * ldt, c, lane, D, acc);
}

// ---------------------------------------------------------------------------
template <typename T, typename ID, bool VEC>
static hipError_t embed_fwd_t(const EmbedPlan& p, const void* ids, const void* table, void* out, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 3) / 4), (unsigned)((p.D + 64 * vec_of<T>() - 1) / (64 * vec_of<T>())));
  embed_fwd_kernel<T, ID, VEC><<<grid, kEmbThreads, 0, s>>>((const ID*)ids, (const T*)table, (T*)out, p.N, p.V, p.D,
                                                            p.ldt, p.ldo, p.scale);
  return hipGetLastError();
}

template <typename ID>
static hipError_t embed_sort(const EmbedPlan& p, const ID* ids, char* ws, uint2** sorted, hipStream_t s) {
  uint2* a = (uint2*)(ws + p.off_pair0);
  uint2* b = (uint2*)(ws + p.off_pair1);
  uint2* seg = (uint2*)(ws + p.off_seg);
  uint32_t* hist = (uint32_t*)(ws + p.off_hist);
  if (p.N <= kCountSort) {
    embed_count_sort<ID><<<(unsigned)((p.N + 63) / 64), 1024, 0, s>>>(ids, a, seg, (int)p.N, p.V, p.padding);
    *sorted = a;
    return hipGetLastError();
  }
  const size_t lds = ((size_t)4 << p.digit);
  for (int k = 0; k < p.passes; ++k) {
    const int shift = k * p.digit;
    if (k == 0) {
      embed_hist<ID, true><<<p.blocks, kEmbThreads, lds, s>>>(ids, nullptr, hist, seg, p.N, p.V, p.padding, shift,
                                                              p.digit, p.rounds);
      embed_scatter<ID, true><<<p.blocks, kEmbThreads, 5 * lds, s>>>(ids, nullptr, a, hist, p.N, p.V, p.padding, shift,
                                                                     p.digit, p.rounds);
    } else {
      embed_hist<ID, false><<<p.blocks, kEmbThreads, lds, s>>>(nullptr, a, hist, nullptr, p.N, p.V, p.padding, shift,
                                                               p.digit, p.rounds);
      embed_scatter<ID, false><<<p.blocks, kEmbThreads, 5 * lds, s>>>(nullptr, a, b, hist, p.N, p.V, p.padding, shift,
                                                                      p.digit, p.rounds);
      uint2* t = a; a = b; b = t;
    }
  }
  *sorted = a;
  return hipGetLastError();
}

template <typename T, bool VEC>
static hipError_t embed_bwd_t(const EmbedPlan& p, const void* ids, const void* dout, char* ws, void* dtable,
                              hipStream_t s) {
  const unsigned slabs = (unsigned)((p.D + 64 * vec_of<T>() - 1) / (64 * vec_of<T>()));
  const int64_t ldp = (p.D + 3) / 4 * 4;
  uint2* sorted = nullptr;
  if (p.N > 0) {
    const hipError_t e = p.id64 ? embed_sort<int64_t>(p, (const int64_t*)ids, ws, &sorted, s)
                                : embed_sort<int32_t>(p, (const int32_t*)ids, ws, &sorted, s);
    if (e != hipSuccess) return e;
    embed_chunks<T, VEC><<<dim3((unsigned)((p.N + kChunk - 1) / kChunk), slabs), 64, 0, s>>>(
        sorted, (uint2*)(ws + p.off_seg), (float*)(ws + p.off_part), (const T*)dout, p.N, p.V, p.D, p.ldo, ldp);
  }
  embed_rows<T, VEC><<<dim3((unsigned)((p.V + 3) / 4), slabs), kEmbThreads, 0, s>>>(
      sorted, (const uint2*)(ws + p.off_seg), (const float*)(ws + p.off_part), (const T*)dout, (T*)dtable, p.V, p.D,
      p.ldo, p.ldt, ldp, p.scale);
  return hipGetLastError();
}

// 16-byte rows: base, stride and length all whole vectors
static bool rows16(const EmbedPlan& p, const void* a, const void* b) {
  const int64_t e = p.dtype == LSTM_F32 ? 4 : 2;
  return aligned16(a) && aligned16(b) && (p.D * e) % 16 == 0 && (p.ldt * e) % 16 == 0 && (p.ldo * e) % 16 == 0;
}

hipError_t launch_embed_fwd(const EmbedPlan& p, const void* ids, const void* table, void* out, hipStream_t s) {
  if (p.N == 0 || p.D == 0) return hipSuccess;
  Timed tm(7, s);
  const bool v = rows16(p, table, out);
#define EMBED_FWD(T)                                                                                         \
  return p.id64 ? (v ? embed_fwd_t<T, int64_t, true>(p, ids, table, out, s)                                  \
                     : embed_fwd_t<T, int64_t, false>(p, ids, table, out, s))                                \
                : (v ? embed_fwd_t<T, int32_t, true>(p, ids, table, out, s)                                  \
                     : embed_fwd_t<T, int32_t, false>(p, ids, table, out, s))
  if (p.dtype == LSTM_F32) EMBED_FWD(float);
  if (p.dtype == LSTM_BF16) EMBED_FWD(bf16_t);
  EMBED_FWD(f16_t);
#undef EMBED_FWD
}

hipError_t launch_embed_bwd(const EmbedPlan& p, const void* ids, const void* dout, char* ws, void* dtable,
                            hipStream_t s) {
  if (p.V == 0 || p.D == 0) return hipSuccess;
  Timed tm(7, s);
  const bool v = rows16(p, dout, dtable);
  if (p.dtype == LSTM_F32)
    return v ? embed_bwd_t<float, true>(p, ids, dout, ws, dtable, s) : embed_bwd_t<float, false>(p, ids, dout, ws, dtable, s);
  if (p.dtype == LSTM_BF16)
    return v ? embed_bwd_t<bf16_t, true>(p, ids, dout, ws, dtable, s) : embed_bwd_t<bf16_t, false>(p, ids, dout, ws, dtable, s);
  return v ? embed_bwd_t<f16_t, true>(p, ids, dout, ws, dtable, s) : embed_bwd_t<f16_t, false>(p, ids, dout, ws, dtable, s);
}

}  // namespace lstm
