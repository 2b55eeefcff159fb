// embed.hip -- token embedding and the gradient of its table (gfx950).
//
//   out[n] = scale * table[ids[n]]        dtable[v] = scale * sum_{ids[n]=v} dout[n]
//
// The forward is a copy of rows.  The gradient brings the tokens of a row
// together in ascending n (so that every call gives the same bits) and writes
// every row once, in one of two ways:
//
// Few tokens (kFew) and a table that one round of work-groups covers: one
// launch.  A work-group owns a run of rows, reads all ids, keeps its own rows'
// tokens in LDS, ordered by a counting sort, and sums them.
//
// Many: a stable radix sort of the tokens by id, the sums of the whole chunks
// of kChunk sorted positions that hold one id alone, and then every row from
// its range of the sorted tokens: the tokens of a chunk that it shares with
// other ids one by one, its whole chunks by their sums.  A row therefore
// costs at most 2 kChunk rows of dout and one sum per chunk, whatever its
// share of the tokens.
//
// Bound by memory: each row of dout is read once and each of dtable written
// once (65536 tokens, 50000 x 1024 bf16: 236 MB in 85 us, 2.8 TB/s: the sort's
// four launches take 22 us of it, the chunks 8, the rows 32, and the gaps
// between six launches most of the rest).  Which way, in us for one launch / the sort, bf16: 4096 tokens of 1000 x 256 9 / 19,
// of 32000 x 512 24 / 30, of 32000 x 1024 37 / 34, of 32000 x 2048 68 / 40;
// 32 tokens of 32000 x 512 21 / 29, of 32000 x 2048 58 / 35: past one round of
// work-groups (kFewGroups of kFewRows rows and a slab) the launch repeats its
// reading of the ids, and the sort wins whatever the number of tokens.
#include "internal.hpp"
#include "seq_internal.hpp"

namespace lstm {

constexpr int kChunk = 64;         // sorted positions per chunk
constexpr int kMaxDigit = 11;      // bits per pass of the sort
constexpr int kFew = 4096;         // tokens the one-launch gradient takes (their list is in LDS),
constexpr int kFewRows = 128, kFewGroups = 512;  // rows per work-group at most, and work-groups
constexpr int kEmbThreads = 256;
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSlab = 512;         // columns of a row a wave holds, 8 per lane

void make_embed_plan(const lstm_embed_shape& s, EmbedPlan* p) {
  p->N = s.N; p->V = s.V; p->D = s.D;
  p->ldt = s.ld_table; p->ldo = s.ld_out; p->padding = s.padding;
  p->scale = s.scale; p->dtype = s.dtype; p->id64 = s.id_type == LSTM_I64;
  p->bits = 1;  // keys 0 .. V, V standing for tokens without a row
  while (((int64_t)1 << p->bits) <= s.V) ++p->bits;
  p->passes = (p->bits + kMaxDigit - 1) / kMaxDigit;
  p->digit = (p->bits + p->passes - 1) / p->passes;
  // every block of the scatter reads the counts of all blocks: at most 128
  p->rounds = 1;
  while ((s.N + kSortThreads * (int64_t)p->rounds - 1) / (kSortThreads * (int64_t)p->rounds) > 128) p->rounds *= 2;
  p->blocks = (int)((s.N + kSortThreads * (int64_t)p->rounds - 1) / (kSortThreads * (int64_t)p->rounds));
  size_t off = 0;
  p->off_pair0 = p->off_pair1 = p->off_hist = p->off_seg = p->off_part = p->total = 0;
  p->few = s.N == 0 || (s.N <= kFew && s.V * ((s.D + kSlab - 1) / kSlab) <= (int64_t)kFewRows * kFewGroups);
  if (p->few) return;
  p->off_pair0 = off; off += align256_seq((size_t)s.N * 8);
  p->off_pair1 = off; off += align256_seq((size_t)s.N * 8);
  p->off_hist = off; off += align256_seq(((size_t)p->blocks << p->digit) * 4);
  p->off_seg = off; off += align256_seq((size_t)s.V * 8);
  p->off_part = off; off += align256_seq((size_t)(s.N / kChunk) * (size_t)((s.D + kSlab - 1) / kSlab * kSlab) * 4);
  p->total = off;
}

// ---------------------------------------------------------------------------
// Slabs of kSlab columns of a row, eight of them per lane: in 16-byte vectors
// 64 lanes side by side where every row is 16-byte aligned (VEC), else one
// by one, 64 apart.
template <typename T, bool VEC>
__device__ __forceinline__ int64_t slab_col(int64_t col0, int lane, int j) {
  constexpr int E = VEC ? vec_of<T>() : 1;
  return col0 + (j / E) * 64 * E + lane * E + j % E;
}
template <typename T, bool VEC>
__device__ __forceinline__ void load_slab(const T* row, int64_t col0, int lane, int64_t D, float* f) {
  if constexpr (VEC) {
    constexpr int E = vec_of<T>();
#pragma unroll
    for (int j = 0; j < 8; j += E) {
      const int64_t c = slab_col<T, VEC>(col0, lane, j);
      u32x4_t v = {0, 0, 0, 0};
      if (c < D) v = *(const u32x4_t*)(row + c);
      unpack<T>(v, f + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t c = slab_col<T, VEC>(col0, lane, j);
      f[j] = c < D ? Elem<T>::load(row + c) : 0.f;
    }
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_slab(T* row, int64_t col0, int lane, int64_t D, const float* f) {
  if constexpr (VEC) {
    constexpr int E = vec_of<T>();
#pragma unroll
    for (int j = 0; j < 8; j += E) {
      const int64_t c = slab_col<T, VEC>(col0, lane, j);
      if (c < D) *(u32x4_t*)(row + c) = pack<T>(f + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t c = slab_col<T, VEC>(col0, lane, j);
      if (c < D) row[c] = Elem<T>::from_f(as_f32(f[j]));
    }
  }
}
__device__ __forceinline__ void clear8(float* f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = 0.f;
}

// Adds the rows of dout at the `m` <= 64 positions that the lanes hold, in
// order, U at a time in flight.
template <typename T, bool VEC, int U>
__device__ __forceinline__ void add_some(uint32_t at, uint32_t i, const T* dout, int64_t ldo, int64_t c, int lane,
                                         int64_t D, float* acc) {
  float f[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u)
    load_slab<T, VEC>(dout + (int64_t)(uint32_t)__builtin_amdgcn_readlane(at, i + u) * ldo, c, lane, D, f[u]);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += f[u][j];
}
template <typename T, bool VEC, int U>
__device__ __forceinline__ void add_rows(uint32_t at, uint32_t m, const T* dout, int64_t ldo, int64_t c, int lane,
                                         int64_t D, float* acc) {
  uint32_t i = 0;
  for (; i + U <= m; i += U) add_some<T, VEC, U>(at, i, dout, ldo, c, lane, D, acc);
  if constexpr (U > 4)
    if (i + 4 <= m) add_some<T, VEC, 4>(at, i, dout, ldo, c, lane, D, acc), i += 4;
  if (i + 2 <= m) add_some<T, VEC, 2>(at, i, dout, ldo, c, lane, D, acc), i += 2;
  if (i < m) add_some<T, VEC, 1>(at, i, dout, ldo, c, lane, D, acc);
}

// ---------------------------------------------------------------------------
// Forward: a wave per (row, slab), bound by memory (65536 rows of 1024 bf16 out
// of 50000: 27 us from the last-level cache, 48 from memory, 185 MB) or, for
// the tokens of one step, by the launch (2.5 us).
template <typename T, typename ID, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) embed_fwd_kernel(const ID* ids, const T* table, T* out, int64_t N,
                                                                int64_t V, int64_t D, int64_t ldt, int64_t ldo,
                                                                float scale) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * 4 + w;
  if (n >= N) return;
  const int64_t id = (int64_t)ids[n];
  const int64_t c = (int64_t)blockIdx.y * kSlab;
  float f[8];
  clear8(f);
  if (id >= 0 && id < V) load_slab<T, VEC>(table + id * ldt, c, lane, D, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] *= scale;
  store_slab<T, VEC>(out + n * ldo, c, lane, D, f);
}

// ---------------------------------------------------------------------------
// Stable ranks inside a wave: the lanes before this one whose `digit` bits of
// d are the same, and how many lanes have them, by one ballot per bit.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, bool real, int digit) {
  uint64_t same = __ballot(real);
  for (int b = 0; b < digit; ++b) {
    const uint64_t one = __ballot((d >> b) & 1);
    same &= ((d >> b) & 1) ? one : ~one;
  }
  return same;
}
// This lane's place among the equal digits of its wave, which `place` counts.
__device__ __forceinline__ uint32_t take_place(volatile uint32_t* place, uint32_t d, bool real, int digit, int lane) {
  const uint64_t same = same_digit(d, real, digit);
  const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
  const uint32_t p = real ? place[d] : 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (real && rank == 0) place[d] = p + __popcll(same);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return p + rank;
}

// ---------------------------------------------------------------------------
// Few tokens: a work-group of 16 waves per (R rows, slab).  Work-group b of n
// owns the rows b, b + n, b + 2 n, ...: in most vocabularies the frequent
// tokens have ids side by side.  A wave sums a row of up to kLight tokens, all
// sixteen together one of more.
constexpr int kFewThreads = 1024, kFewWaves = 16, kLight = 16;

template <typename T, typename ID, bool VEC>
__global__ void __launch_bounds__(kFewThreads) embed_few(const ID* ids, const T* dout, T* dtable, int N, int64_t V,
                                                         int64_t D, int64_t ldo, int64_t ldt, int64_t padding,
                                                         float scale, int R, int rbits) {
  constexpr int kRounds = kFew / kFewThreads;
  __shared__ uint32_t list[kFew];                      // this run's tokens, by row, then n
  __shared__ uint32_t place[kFewWaves][kFewRows], start[kFewRows + 1];
  __shared__ float part[kFewWaves][kSlab];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t nb = gridDim.x, me = blockIdx.x;
  const int64_t c = (int64_t)blockIdx.y * kSlab;
  const int rows = (int)(((uint32_t)V - me + nb - 1) / nb);  // <= R
  // each wave a stretch of the tokens, 64 a round
  const int rounds = (N + kFewThreads - 1) / kFewThreads;
  int64_t id[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int n = (w * rounds + k) * 64 + lane;
    id[k] = k < rounds && n < N ? (int64_t)ids[n] : -1;
  }
  for (int i = tid; i < kFewWaves * kFewRows; i += kFewThreads) (&place[0][0])[i] = 0;
  __syncthreads();
  uint32_t row[kRounds];  // R: none
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const bool any = id[k] >= 0 && id[k] < V && id[k] != padding;
    const uint32_t v = any ? (uint32_t)id[k] : 0, r = v / nb;
    row[k] = any && v - r * nb == me ? r : (uint32_t)R;
    if (row[k] < (uint32_t)R) atomicAdd(&place[w][row[k]], 1u);
  }
  __syncthreads();
  if (w == 0) {  // the rows' first places, two rows a lane
    uint32_t n0 = 0, n1 = 0;
    for (int k = 0; k < kFewWaves; ++k) {
      n0 += place[k][2 * lane];
      n1 += place[k][2 * lane + 1];
    }
    uint32_t inc = n0 + n1;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t up = __shfl_up(inc, o);
      if (lane >= o) inc += up;
    }
    start[2 * lane + 1] = inc - n1;
    start[2 * lane + 2] = inc;
    if (lane == 0) start[0] = 0;
  }
  __syncthreads();
  if (tid < kFewRows) {
    uint32_t p = start[tid];
    for (int k = 0; k < kFewWaves; ++k) {
      const uint32_t n = place[k][tid];
      place[k][tid] = p;
      p += n;
    }
  }
  __syncthreads();
  if (start[kFewRows] > 0) {
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const bool real = row[k] < (uint32_t)R;
      if (!__ballot(real)) continue;
      const uint32_t at = take_place(place[w], real ? row[k] : 0, real, rbits, lane);
      if (real) list[at] = (uint32_t)((w * rounds + k) * 64 + lane);
    }
  }
  __syncthreads();
  // a wave per row; rows of many tokens by all waves, each a sixteenth
  for (int r = w; r < rows; r += kFewWaves) {
    const uint32_t lo = start[r], n = start[r + 1] - lo;
    if (n > kLight) continue;
    float acc[8];
    clear8(acc);
    add_rows<T, VEC, 8>((uint32_t)lane < n ? list[lo + lane] : 0, n, dout, ldo, c, lane, D, acc);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] *= scale;
    store_slab<T, VEC>(dtable + ((int64_t)r * nb + me) * ldt, c, lane, D, acc);
  }
  for (int r = 0; r < rows; ++r) {
    const uint32_t lo = start[r], n = start[r + 1] - lo;
    if (n <= kLight) continue;
    const uint32_t each = (n + kFewWaves - 1) / kFewWaves;
    const uint32_t a = lo + w * each < lo + n ? lo + w * each : lo + n, b = a + each < lo + n ? a + each : lo + n;
    float acc[8];
    clear8(acc);
    for (uint32_t p = a; p < b; p += 64) {
      const uint32_t m = b - p < 64 ? b - p : 64;
      add_rows<T, VEC, 8>((uint32_t)lane < m ? list[p + lane] : 0, m, dout, ldo, c, lane, D, acc);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) part[w][j * 64 + lane] = acc[j];
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float sum = 0.f;
        for (int k = 0; k < kFewWaves; ++k) sum += part[k][j * 64 + lane];
        acc[j] = sum * scale;
      }
      store_slab<T, VEC>(dtable + ((int64_t)r * nb + me) * ldt, c, lane, D, acc);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The sort.  Key of a token: its id, or V where it has no gradient.
template <typename ID>
__device__ __forceinline__ uint32_t key_of(const ID* ids, int64_t n, int64_t V, int64_t padding) {
  const int64_t id = (int64_t)ids[n];
  return (uint32_t)(id >= 0 && id < V && id != padding ? id : V);
}

// Digit counts of each block's tokens.  In the first pass the rows' ranges
// start empty here, with the help of work-groups past the blocks where there
// are few tokens and many rows.
template <typename ID, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) embed_hist(const ID* ids, const uint2* in, uint32_t* hist, uint2* seg,
                                                           int64_t N, int64_t V, int64_t padding, int shift, int digit,
                                                           int rounds, int blocks) {
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  uint32_t* cnt = (uint32_t*)lds_raw;
  const int bins = 1 << digit, tid = threadIdx.x;
  for (int b = tid; b < bins; b += kSortThreads) cnt[b] = 0;
  if (FIRST) {
    const int64_t all = (int64_t)gridDim.x * kSortThreads;
    for (int64_t i = (int64_t)blockIdx.x * kSortThreads + tid; i < V; i += all) seg[i] = make_uint2(0, 0);
    if ((int)blockIdx.x >= blocks) return;
  }
  __syncthreads();
  const int64_t n0 = (int64_t)blockIdx.x * kSortThreads * rounds;
  for (int r = 0; r < rounds; ++r) {
    const int64_t n = n0 + r * kSortThreads + tid;
    if (n < N) {
      const uint32_t k = FIRST ? key_of(ids, n, V, padding) : in[n].x;
      atomicAdd(&cnt[(k >> shift) & (bins - 1)], 1u);
    }
  }
  __syncthreads();
  for (int b = tid; b < bins; b += kSortThreads) hist[((int64_t)blockIdx.x << digit) + b] = cnt[b];
}

// Stable scatter by one digit: the first place of a digit in a block is the
// number of tokens of lower digits plus that of the digit in the blocks
// before; a wave's tokens follow those of the waves before it.
template <typename ID, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) embed_scatter(const ID* ids, const uint2* in, uint2* out,
                                                              const uint32_t* hist, int64_t N,
                                                              int64_t V, int64_t padding, int shift, int digit,
                                                              int rounds) {
  extern __shared__ __attribute__((aligned(16))) char lds_raw[];
  const int bins = 1 << digit, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  uint32_t* first = (uint32_t*)lds_raw;   // [bins] counts, then first places
  uint32_t* start = first + bins;         // [bins] this block's offset inside a digit
  uint32_t* wave = start + bins;          // [kSortWaves][bins]
  __shared__ uint32_t wsum[kSortWaves];
  const int64_t n0 = (int64_t)blockIdx.x * kSortThreads * rounds + (int64_t)w * 64 * rounds;
  auto token = [&](int64_t n) {
    uint2 t = make_uint2(0, (uint32_t)n);
    if (n < N) {
      if constexpr (FIRST) t.x = key_of(ids, n, V, padding);
      else t = in[n];
    }
    return t;
  };
  const uint2 t0 = token(n0 + lane);  // in flight beside the counts
  for (int b = tid; b < kSortWaves * bins; b += kSortThreads) wave[b] = 0;
  // totals of every digit, and this block's offset inside it: up to `share`
  // threads a digit, each over every share-th block (at most 32 loads, all in
  // flight), their sums joined in LDS
  const int share = bins < kSortThreads ? kSortThreads / bins : 1;
  for (int b = tid; b < bins; b += kSortThreads) first[b] = start[b] = 0;
  __syncthreads();
  for (int i = tid; i < bins * share; i += kSortThreads) {
    const int b = i & (bins - 1);
    uint32_t total = 0, before = 0;
#pragma unroll 16
    for (int k = i >> digit; k < (int)gridDim.x; k += share) {
      const uint32_t c = hist[((int64_t)k << digit) + b];
      if (k < (int)blockIdx.x) before += c;
      total += c;
    }
    atomicAdd(&first[b], total);
    atomicAdd(&start[b], before);
  }
  __syncthreads();
  // exclusive sum over the digits, one or two side by side per thread
  const int run = bins > kSortThreads ? 2 : 1;
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
      const uint32_t c = first[tid * run + b];
      first[tid * run + b] = at;
      at += c;
    }
  // the waves' digit counts
  for (int r = 0; r < rounds; ++r) {
    const int64_t n = n0 + r * 64 + lane;
    if (n < N) atomicAdd(&wave[w * bins + (((r == 0 ? t0 : token(n)).x >> shift) & (bins - 1))], 1u);
  }
  __syncthreads();
  // their first places
  for (int b = tid; b < bins; b += kSortThreads) {
    uint32_t p = first[b] + start[b];
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) {
      const uint32_t c = wave[k * bins + b];
      wave[k * bins + b] = p;
      p += c;
    }
  }
  __syncthreads();
  for (int r = 0; r < rounds; ++r) {
    const int64_t n = n0 + r * 64 + lane;
    const bool real = n < N;
    const uint2 t = r == 0 ? t0 : token(n);
    const uint32_t p = take_place(wave + w * bins, (t.x >> shift) & (bins - 1), real, digit, lane);
    if (real) out[p] = t;
  }
}

// ---------------------------------------------------------------------------
// Adds the rows of dout at sorted positions [lo, hi), in order.
template <typename T, bool VEC, int U>
__device__ __forceinline__ void sum_rows(const uint2* sorted, uint32_t lo, uint32_t hi, const T* dout, int64_t ldo,
                                         int64_t c, int lane, int64_t D, float* acc) {
  for (uint32_t p = lo; p < hi; p += 64) {
    const uint32_t m = hi - p < 64 ? hi - p : 64;
    add_rows<T, VEC, U>((uint32_t)lane < m ? sorted[p + lane].y : 0, m, dout, ldo, c, lane, D, acc);
  }
}

// A wave per (chunk, slab): the ranges of the ids that start or end in the
// chunk, and the sum of a chunk of one id (eight values of a lane side by
// side).
template <typename T, bool VEC>
__global__ void __launch_bounds__(64) embed_chunks(const uint2* sorted, uint2* seg, float* part, const T* dout,
                                                   int64_t N, int64_t V, int64_t D, int64_t ldo, int64_t ldp) {
  const int lane = threadIdx.x;
  const int64_t p0 = (int64_t)blockIdx.x * kChunk, p = p0 + lane;
  const uint2 me = p < N ? sorted[p] : make_uint2((uint32_t)V, 0);
  const uint32_t key = me.x;
  if (blockIdx.y == 0 && key < (uint32_t)V) {
    if (p == 0 || sorted[p - 1].x != key) seg[key].x = (uint32_t)p;
    if (p + 1 == N || sorted[p + 1].x != key) seg[key].y = (uint32_t)(p + 1);
  }
  const uint32_t k0 = __builtin_amdgcn_readlane(key, 0), k1 = __builtin_amdgcn_readlane(key, 63);
  if (k0 != k1 || k0 == (uint32_t)V) return;
  const int64_t c = (int64_t)blockIdx.y * kSlab;
  float acc[8];
  clear8(acc);
  add_rows<T, VEC, 16>(me.y, kChunk, dout, ldo, c, lane, D, acc);
  float* o = part + (int64_t)blockIdx.x * ldp + c + lane * 8;
#pragma unroll
  for (int j = 0; j < 8; j += 4) *(f32x4_t*)(o + j) = f32x4_t{acc[j], acc[j + 1], acc[j + 2], acc[j + 3]};
}

// A wave per (row of dtable, slab).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) embed_rows(const uint2* sorted, const uint2* seg, const float* part,
                                                          const T* dout, T* dtable, int64_t V, int64_t D, int64_t ldo,
                                                          int64_t ldt, int64_t ldp, float scale) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t v = (int64_t)blockIdx.x * 4 + w;
  if (v >= V) return;
  const int64_t c = (int64_t)blockIdx.y * kSlab;
  float acc[8];
  clear8(acc);
  const uint2 sg = seg[v];
  const uint32_t lo = __builtin_amdgcn_readfirstlane(sg.x), hi = __builtin_amdgcn_readfirstlane(sg.y);
  // [lo, a) rows, whole chunks [a, b), [b, hi) rows
  uint32_t a = (lo + kChunk - 1) / kChunk * kChunk, b = hi / kChunk * kChunk;
  if (a > hi) a = hi;
  if (b < a) b = a;
  sum_rows<T, VEC, 4>(sorted, lo, a, dout, ldo, c, lane, D, acc);
#pragma unroll 4
  for (uint32_t k = a / kChunk; k < b / kChunk; ++k) {
    const float* q = part + (int64_t)k * ldp + c + lane * 8;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const f32x4_t x = *(const f32x4_t*)(q + j);
      acc[j] += x[0]; acc[j + 1] += x[1]; acc[j + 2] += x[2]; acc[j + 3] += x[3];
    }
  }
  sum_rows<T, VEC, 4>(sorted, b, hi, dout, ldo, c, lane, D, acc);
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] *= scale;
  store_slab<T, VEC>(dtable + v * ldt, c, lane, D, acc);
}

// ---------------------------------------------------------------------------
static unsigned slabs_of(int64_t D) { return (unsigned)((D + kSlab - 1) / kSlab); }

template <typename T, typename ID, bool VEC>
static hipError_t embed_fwd_t(const EmbedPlan& p, const void* ids, const void* table, void* out, hipStream_t s) {
  for (int64_t n0 = 0; n0 < p.N; n0 += 4 * kMaxGroups) {
    const int64_t N = p.N - n0 < 4 * kMaxGroups ? p.N - n0 : 4 * kMaxGroups;
    embed_fwd_kernel<T, ID, VEC><<<dim3((unsigned)((N + 3) / 4), slabs_of(p.D)), kEmbThreads, 0, s>>>(
        (const ID*)ids + n0, (const T*)table, (T*)out + n0 * p.ldo, N, p.V, p.D, p.ldt, p.ldo, p.scale);
  }
  return hipGetLastError();
}

template <typename ID>
static hipError_t embed_sort(const EmbedPlan& p, const ID* ids, char* ws, uint2** sorted, hipStream_t s) {
  uint2* a = (uint2*)(ws + p.off_pair0);
  uint2* b = (uint2*)(ws + p.off_pair1);
  uint2* seg = (uint2*)(ws + p.off_seg);
  uint32_t* hist = (uint32_t*)(ws + p.off_hist);
  const size_t lds = (size_t)4 << p.digit, lds_all = lds * (2 + kSortWaves);
  if (lds_all > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute((const void*)embed_scatter<ID, true>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)lds_all);
    if (e == hipSuccess)
      e = hipFuncSetAttribute((const void*)embed_scatter<ID, false>, hipFuncAttributeMaxDynamicSharedMemorySize,
                              (int)lds_all);
    if (e != hipSuccess) return e;
  }
  for (int k = 0; k < p.passes; ++k) {
    const int shift = k * p.digit;
    if (k == 0) {
      const int64_t clear = p.V / (4 * kSortThreads) < 512 ? p.V / (4 * kSortThreads) : 512;
      const unsigned grid = (unsigned)(clear > p.blocks ? clear : p.blocks);
      embed_hist<ID, true><<<grid, kSortThreads, lds, s>>>(ids, nullptr, hist, seg, p.N, p.V, p.padding, shift, p.digit,
                                                           p.rounds, p.blocks);
      embed_scatter<ID, true><<<p.blocks, kSortThreads, lds_all, s>>>(ids, nullptr, a, hist, p.N, p.V, p.padding, shift,
                                                                      p.digit, p.rounds);
    } else {
      embed_hist<ID, false><<<p.blocks, kSortThreads, lds, s>>>(nullptr, a, hist, nullptr, p.N, p.V, p.padding, shift,
                                                                p.digit, p.rounds, p.blocks);
      embed_scatter<ID, false><<<p.blocks, kSortThreads, lds_all, s>>>(nullptr, a, b, hist, p.N, p.V, p.padding, shift,
                                                                       p.digit, p.rounds);
      uint2* t = a; a = b; b = t;
    }
  }
  *sorted = a;
  return hipGetLastError();
}

template <typename T, typename ID, bool VEC>
static hipError_t embed_bwd_t(const EmbedPlan& p, const void* ids, const void* dout, char* ws, void* dtable,
                              hipStream_t s) {
  const unsigned slabs = slabs_of(p.D);
  if (p.few) {
    int64_t R = (p.V * slabs + kFewGroups - 1) / kFewGroups;  // two work-groups a compute unit
    R = R < 16 ? 16 : R > kFewRows ? kFewRows : (R + 15) / 16 * 16;
    int rbits = 4;
    while ((1 << rbits) < R) ++rbits;
    embed_few<T, ID, VEC><<<dim3((unsigned)((p.V + R - 1) / R), slabs), kFewThreads, 0, s>>>(
        (const ID*)ids, (const T*)dout, (T*)dtable, (int)p.N, p.V, p.D, p.ldo, p.ldt, p.padding, p.scale, (int)R, rbits);
    return hipGetLastError();
  }
  const int64_t ldp = (int64_t)slabs * kSlab;
  uint2* sorted = nullptr;
  const hipError_t e = embed_sort<ID>(p, (const ID*)ids, ws, &sorted, s);
  if (e != hipSuccess) return e;
  embed_chunks<T, VEC><<<dim3((unsigned)((p.N + kChunk - 1) / kChunk), slabs), 64, 0, s>>>(
      sorted, (uint2*)(ws + p.off_seg), (float*)(ws + p.off_part), (const T*)dout, p.N, p.V, p.D, p.ldo, ldp);
  for (int64_t v0 = 0; v0 < p.V; v0 += 4 * kMaxGroups) {
    const int64_t V = p.V - v0 < 4 * kMaxGroups ? p.V - v0 : 4 * kMaxGroups;
    embed_rows<T, VEC><<<dim3((unsigned)((V + 3) / 4), slabs), kEmbThreads, 0, s>>>(
        sorted, (const uint2*)(ws + p.off_seg) + v0, (const float*)(ws + p.off_part), (const T*)dout,
        (T*)dtable + v0 * p.ldt, V, p.D, p.ldo, p.ldt, ldp, p.scale);
  }
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
#define EMBED_BWD(T)                                                                                         \
  return p.id64 ? (v ? embed_bwd_t<T, int64_t, true>(p, ids, dout, ws, dtable, s)                            \
                     : embed_bwd_t<T, int64_t, false>(p, ids, dout, ws, dtable, s))                          \
                : (v ? embed_bwd_t<T, int32_t, true>(p, ids, dout, ws, dtable, s)                            \
                     : embed_bwd_t<T, int32_t, false>(p, ids, dout, ws, dtable, s))
  if (p.dtype == LSTM_F32) EMBED_BWD(float);
  if (p.dtype == LSTM_BF16) EMBED_BWD(bf16_t);
  EMBED_BWD(f16_t);
#undef EMBED_BWD
}

}  // namespace lstm
