// attend.hip -- cross attention forward (gfx950).
//
//   s = scale q . k over the valid keys,  p = exp(s - lse),  o = sum p v
//
// A wave holds 32 query rows (attend_common.hpp) as one operand in registers
// and walks over tiles of keys in LDS: S^T = K Q^T leaves row r of the tile's
// scores down one lane's registers (and those of lane ^ 32), so the softmax
// statistics are sums over a lane's own registers, and the rounded p are the
// second operand of O^T += V^T P^T as they stand; neither S nor P touches
// memory.  Scores are kept in powers of two, y = s log2 e - m, against a
// reference m that moves only when a score passes it by more than kMaxLag
// (2^kMaxLag times the largest p is no loss of precision in floating point);
// most tiles rescale nothing.  In fp16 the reference stays kLift below the
// largest score seen, so that p, as an operand, is a normal number down to
// 2^-21 of the largest and not 2^-14.
//
// Two kernels.  attend_fwd_kernel: four waves of 32 rows share each tile of
// keys, double-buffered, one barrier a tile; the matrix products are the
// bound (8 sequences, 32/8 heads of 128, 1024 x up to 4096 keys, bf16: 340-355
// us, 980 TFLOP/s; 64 sequences, 16 heads of 64, 256 x 256: 36 us, 3.0 TB/s of
// its valid rows and no unit's bound: matrix units 14 % busy, vector units 40 %,
// each wave's loop at most four tiles).  attend_step_kernel: for few rows (one token of each sequence):
// every wave walks over its own tiles with no barrier, the keys split over the
// waves and over `splits` work-groups, joined at the end; the keys' and
// values' bytes are the bound (see the kernel).
#include <type_traits>

#include "attend_common.hpp"

namespace lstm {

template <typename T> constexpr float kLift = std::is_same<T, f16_t>::value ? 7.f : 0.f;
template <typename T> constexpr float kMaxLag = 8.f + kLift<T>;  // fp16: p up to 2^15
constexpr int kAheadRows = 8, kAheadCols = 4;  // fragments read ahead of their products

// One tile of 32 KT keys for a wave's 32 rows.
template <typename T, int DP, int KT>
__device__ __forceinline__ void attend_tile(const char* kt, const char* vt, uint64_t bits, const u32x4_t* q, f32x16_t* o,
                                            float& m, float& l, float c2, int lane) {
  using TL = Tile<T, DP>;
  lane = tile_lane<DP == 256 || (sizeof(T) == 4 && DP == 128)>(lane);
  f32x16_t s[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) s[t] = zero16();
  // fragment f of the keys: subtile f / KB, k-block f % KB; of the values:
  // k-block f / (DP / 32) of the rows, d-tile f % (DP / 32)
  constexpr int NDT = DP / 32;
  Ahead<KT * TL::KB, kAheadRows> ak;
  Ahead<KT * TL::PB * NDT, kAheadCols> av;
  auto read_k = [&](int f) { return TL::row_frag(kt, 32 * (f / TL::KB), f % TL::KB, lane); };
  auto read_v = [&](int f) { return TL::col_frag(vt, TL::KR * (f / NDT), f % NDT, lane); };
  ak.start(read_k);
  ak.run(read_k, [&](int f, u32x4_t a) { s[f / TL::KB] = Mm<T>::mac(a, q[f % TL::KB], s[f / TL::KB]); });
  av.start(read_v);
  constexpr uint64_t kAll = KT == 2 ? ~(uint64_t)0 : 0xffffffffull;
  if ((bits & kAll) != kAll) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const uint32_t mine = (uint32_t)(bits >> (32 * t)) >> (4 * (lane >> 5));
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!((mine >> reg_row(i, 0)) & 1)) s[t][i] = -INFINITY;
    }
  }
  float top = s[0][0];
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
  top = fmaxf(top, other_half(top)) * c2;
  if (__ballot(top > m + kMaxLag<T>)) {
    const float to = fmaxf(m, top - kLift<T>), by = to == m ? 1.f : __builtin_amdgcn_exp2f(m - to);
    m = to;
    l *= by;
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[dt][i] *= by;
  }
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[t][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], c2, -ref));
      l += s[t][i];
    }
  u32x4_t p[KT * TL::PB];
#pragma unroll
  for (int i = 0; i < KT * TL::PB; ++i) p[i] = TL::reg_frag(s[i / TL::PB], i % TL::PB);
  av.run(read_v, [&](int f, u32x4_t a) { o[f % NDT] = Mm<T>::mac(a, p[f / NDT], o[f % NDT]); });
}

// Keys per tile of the shared kernel: two double-buffered tiles within 128 KB.
template <typename T, int DP> constexpr int fwd_keys() { return 4 * 64 * Tile<T, DP>::C * 16 <= 128 * 1024 ? 64 : 32; }

// Two waves a SIMD but for rows of 512 bytes and more: q, o and s alone are
// 224 registers there (bf16 heads of 256, 16 sequences, 16/8 heads, 512 x 512:
// two waves, spilled, 548 us, one 131).
template <typename T, int DP, bool DMA>
__global__ void __launch_bounds__(256, DP * sizeof(T) >= 512 ? 1 : 2) attend_fwd_kernel(AttendArgs a) {
  using TL = Tile<T, DP>;
  constexpr int NK = fwd_keys<T, DP>(), TB = NK * TL::C * 16;
  extern __shared__ __attribute__((aligned(16))) char lds[];  // K, V tiles, twice
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int grp, tile;
  if (!group_of(a, blockIdx.x, &grp, &tile)) return;
  const int b = grp / a.Hk, hk = grp - b * a.Hk;
  const int end = keys_of(a, b);
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_b : nullptr;
  const uint32_t r = (uint32_t)tile * 128 + w * 32 + (lane & 31);
  const bool ok = r < a.M;
  const uint32_t t = r / a.G, h = hk * a.G + (r - t * a.G);

  u32x4_t q[TL::KB];
  load_row_frags<T, DP>((const T*)a.q + t * a.qs.t + b * a.qs.b + h * a.qs.h, a.D, a.whole & kWholeQ, ok, lane, q);
  Loader<T, DP, NK, 4, DMA> lk, lv;
  lk.init((const T*)a.k + b * a.ks.b + hk * a.ks.h, a.ks.t, a.D, a.whole & kWholeK, mask, w, lane);
  lv.init((const T*)a.v + b * a.vs.b + hk * a.vs.h, a.vs.t, a.D, a.whole & kWholeV, mask, w, lane);

  f32x16_t o[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) o[dt] = zero16();
  float m = -INFINITY, l = 0.f;
  const float c2 = a.scale * kLog2e;
  const int n = (end + NK - 1) / NK;
  if (n > 0) {
    lk.load(0, end, lds);
    lv.load(0, end, lds + TB);
  }
  uint64_t bits = key_bits(mask, 0, end, lane);
  for (int i = 0; i < n; ++i) {
    wait_vmem();
    __syncthreads();
    char* cur = lds + (i & 1) * 2 * TB;
    char* nxt = lds + (~i & 1) * 2 * TB;
    const uint64_t now = bits;
    if (i + 1 < n) {
      lk.load((i + 1) * NK, end, nxt);
      lv.load((i + 1) * NK, end, nxt + TB);
      bits = key_bits(mask, (i + 1) * NK, end, lane);
    }
    attend_tile<T, DP, NK / 32>(cur, cur + TB, now, q, o, m, l, c2, lane);
  }
  l += other_half(l);
  if (!ok) return;
  const float by = l == 0.f ? 0.f : 1.f / l;
  store_col<T, DP>((T*)a.out + t * a.os.t + b * a.os.b + h * a.os.h, o, by, a.D, a.whole & kWholeO, lane);
  if (lane < 32) a.lse[((int64_t)b * a.Hq + h) * a.Tq + t] = kLn2 * (m + __builtin_amdgcn_logf(l));
}

// ---------------------------------------------------------------------------
// Few rows (step_waves in attend_common.hpp): the keys' tiles dealt to the
// waves, the waves' parts joined in LDS.  One tile a wave and eight waves, of
// which the others' loads are in flight while one computes: 16 sequences, 16
// heads of 128, one row x up to 512 keys, bf16 14.1 us (42 MB); 8 sequences,
// 32/8 heads, up to 32768 keys, fp16 143 us (671 MB, 4.7 TB/s); with two tiles
// a wave and four waves 16.8 and 145-151 us.
template <typename T, int DP, bool DMA>
__global__ void __launch_bounds__((64 * step_waves<T, DP>()), 1) attend_step_kernel(AttendArgs a) {
  using TL = Tile<T, DP>;
  constexpr int NW = step_waves<T, DP>(), TB = TL::kBytes32;
  extern __shared__ __attribute__((aligned(16))) char lds[];  // per wave: K, V tile
  __shared__ float wm[NW][32], wl[NW][32];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int grp, tile;
  if (!group_of(a, blockIdx.x, &grp, &tile)) return;
  const int rt = tile / a.splits, sp = tile - rt * a.splits;
  const int b = grp / a.Hk, hk = grp - b * a.Hk;
  const int end = keys_of(a, b);
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_b : nullptr;
  const uint32_t r = (uint32_t)rt * 32 + (lane & 31);
  const bool ok = r < a.M;
  const uint32_t t = r / a.G, h = hk * a.G + (r - t * a.G);

  u32x4_t q[TL::KB];
  load_row_frags<T, DP>((const T*)a.q + t * a.qs.t + b * a.qs.b + h * a.qs.h, a.D, a.whole & kWholeQ, ok, lane, q);
  Loader<T, DP, 32, 1, DMA> lk, lv;
  lk.init((const T*)a.k + b * a.ks.b + hk * a.ks.h, a.ks.t, a.D, a.whole & kWholeK, mask, 0, lane);
  lv.init((const T*)a.v + b * a.vs.b + hk * a.vs.h, a.vs.t, a.D, a.whole & kWholeV, mask, 0, lane);
  char* mine = lds + w * 2 * TB;

  f32x16_t o[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) o[dt] = zero16();
  float m = -INFINITY, l = 0.f;
  const float c2 = a.scale * kLog2e;
  // this sequence's tiles in equal shares; the waves take theirs in turn
  const int all = (end + 31) / 32, each = (all + a.splits - 1) / a.splits;
  const int first = sp * each + w, last = (sp + 1) * each < all ? (sp + 1) * each : all;
  uint64_t bits = 0;
  if (first < last) {
    lk.load(first * 32, end, mine);
    lv.load(first * 32, end, mine + TB);
    bits = key_bits(mask, first * 32, end, lane);
  }
  for (int i = first; i < last; i += NW) {
    const uint64_t now = bits;
    wait_vmem();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    attend_tile<T, DP, 1>(mine, mine + TB, now, q, o, m, l, c2, lane);
    if (i + NW < last) {
      __builtin_amdgcn_s_waitcnt(kLgkm0);  // every fragment of this tile is read
      lk.load((i + NW) * 32, end, mine);
      lv.load((i + NW) * 32, end, mine + TB);
      bits = key_bits(mask, (i + NW) * 32, end, lane);
    }
  }
  l += other_half(l);
  // the waves' parts on one reference: column r of wave w at its own stages
  float* mo = (float*)mine;  // [DP][32]
  __syncthreads();
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) mo[(32 * dt + reg_row(i, lane)) * 32 + (lane & 31)] = o[dt][i];
  if (lane < 32) {
    wm[w][lane] = m;
    wl[w][lane] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f, by[NW];
#pragma unroll
  for (int k = 0; k < NW; ++k) top = fmaxf(top, wm[k][lane & 31]);
  const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    by[k] = __builtin_amdgcn_exp2f(wm[k][lane & 31] - ref);
    sum += wl[k][lane & 31] * by[k];
  }
  if (!ok) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t unit = ((int64_t)grp * (a.tiles / a.splits) + rt) * a.splits + sp;
  T* out = (T*)a.out + t * a.os.t + b * a.os.b + h * a.os.h;
  float* part = a.part + (unit * 32 + (lane & 31)) * a.D;
  for (int d = 2 * w + (lane >> 5); d < a.D; d += 2 * NW) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) v += ((const float*)(lds + k * 2 * TB))[d * 32 + (lane & 31)] * by[k];
    if (a.splits == 1) out[d] = Elem<T>::from_f(as_f32(v * inv));
    else part[d] = v;
  }
  if (w == 0 && lane < 32) {
    if (a.splits == 1) {
      a.lse[((int64_t)b * a.Hq + h) * a.Tq + t] = kLn2 * (top + __builtin_amdgcn_logf(sum));
    } else {
      a.part_ml[2 * (unit * 32 + lane)] = top;
      a.part_ml[2 * (unit * 32 + lane) + 1] = sum;
    }
  }
}

// A wave per row: the parts of its keys, their statistics in one lane each and
// their outputs read side by side (256 rows of 128 values: 5.4 us; lanes that
// walked over the statistics one by one took 49 for 32 parts).
template <typename T>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendArgs a, int row_tiles) {
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t n = (int64_t)a.B * a.Hk * a.M;
  if (i >= n) return;
  const int64_t grp = i / a.M;
  const uint32_t r = (uint32_t)(i - grp * a.M), t = r / a.G;
  const int b = (int)(grp / a.Hk);
  const uint32_t h = (uint32_t)(grp - (int64_t)b * a.Hk) * a.G + (r - t * a.G);
  const int64_t unit = ((grp * row_tiles + r / 32) * a.splits) * 32 + (r & 31);  // + 32 per part
  // lane k: part k's statistics (at most 64 parts)
  float m = -INFINITY, l = 0.f;
  if (lane < a.splits) {
    m = a.part_ml[2 * (unit + 32 * lane)];
    l = a.part_ml[2 * (unit + 32 * lane) + 1];
  }
  float top = m;
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float by = __builtin_amdgcn_exp2f(m - (top == -INFINITY ? 0.f : top));
  float sum = l * by;
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* out = (T*)a.out + t * a.os.t + b * a.os.b + h * a.os.h;
  for (int d0 = 0; d0 < a.D; d0 += 64) {
    const int d = d0 + lane;
    const float* from = a.part + unit * a.D + (d < a.D ? d : 0);
    float v = 0.f;
    for (int k0 = 0; k0 < a.splits; k0 += 8) {  // eight loads in flight
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = k0 + k < a.splits ? from[(int64_t)32 * (k0 + k) * a.D] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v += x[k] * __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(by), (k0 + k) & 63));
    }
    if (d < a.D) out[d] = Elem<T>::from_f(as_f32(v * inv));
  }
  if (lane == 0) a.lse[((int64_t)b * a.Hq + h) * a.Tq + t] = kLn2 * (top + __builtin_amdgcn_logf(sum));
}

// ---------------------------------------------------------------------------
void make_attend_plan(const lstm_attend_shape& s, int cus, AttendPlan* p) {
  p->dtype = s.dtype;
  const int dps[6] = {32, 64, 96, 128, 192, 256};
  p->DP = 256;
  for (int i = 5; i >= 0; --i)
    if (s.D <= dps[i]) p->DP = dps[i];
  const int64_t e = s.dtype == LSTM_F32 ? 4 : 2, G = s.Hk > 0 ? s.Hq / s.Hk : 1, M = s.Tq * G, groups = s.B * s.Hk;
  p->row_tiles32 = (int)((M + 31) / 32);
  // The shared kernels where their work-groups fill at least half the device.
  // 128 rows x 1024 keys in bf16, step kernel / shared, us, for 64, 96, 128,
  // 192 and 256 pairs of a sequence and a key head: heads of 64 20 / 21, 26 /
  // 21, 17 / 21, 24 / 21, 29 / 22; of 128 16 / 27, 28 / 28, 28 / 28, 41 / 29,
  // 52 / 30; the backward by the same rule 30 / 40, 46 / 46, 51 / 51, 75 / 63,
  // 91 / 72 and 46 / 59, 77 / 73, 84 / 79, 123 / 102, 159 / 124; dk and dv of
  // 1024 rows x 128 keys 28 / 41, 42 / 45, 49 / 52, 69 / 61, 87 / 71.  Up to 32
  // rows a pair fill a wave at most: 1024 pairs 53 / 55, of 48 rows 72 / 58.
  p->step = M <= 32 || groups * ((M + 127) / 128) < cus / 2;
  p->few_rows = p->step;
  p->few_keys = groups * ((s.Tk + 127) / 128) < cus / 2;
  p->splits = 1;
  if (p->step && groups > 0 && M > 0) {
    // fill the device, or, with long keys, twice that, which evens out
    // sequences of different lengths; never less than two tiles a wave (the
    // join costs a launch).  One token, 8 key heads of 128 shared by four, us,
    // one part / this rule / others: 2 sequences of 2048 keys 19 / 16 / two
    // parts 18; 4 of 16384 100 / 44 / two 64, sixteen 48; 32 of 2048 38 / 39 /
    // four 50; 32 of 8192 160 / 157 / eight 171.
    const int64_t units = groups * p->row_tiles32, tile = 2 * 32 * p->DP * e;
    const int64_t waves = step_waves_of(tile), keys = 32 * waves;
    const int64_t fill = (cus * (waves * tile <= 80 * 1024 ? 2 : 1) + units - 1) / units;
    int64_t n = s.Tk / (8 * keys) < 2 * fill ? s.Tk / (8 * keys) : 2 * fill;
    if (n < fill) n = fill;
    if (n > s.Tk / (2 * keys)) n = s.Tk / (2 * keys);
    if (n > 64) n = 64;
    if (n < 1) n = 1;
    p->splits = (int)n;
  }
  size_t off = 0;
  p->off_part = p->off_ml = 0;
  if (p->splits > 1) {
    const size_t rows = (size_t)groups * p->row_tiles32 * p->splits * 32;
    p->off_part = off; off += align256_seq(rows * (size_t)s.D * 4);
    p->off_ml = off; off += align256_seq(rows * 8);
  }
  p->total_fwd = off;
  p->total_bwd = align256_seq((size_t)s.B * s.Hq * s.Tq * 8);
}

template <typename T, int DP, bool DMA>
static hipError_t attend_fwd_t(const AttendPlan& p, const AttendArgs& a0, hipStream_t s) {
  AttendArgs a = a0;
  constexpr int C = Tile<T, DP>::C;
  if (p.step) {
    constexpr int NW = step_waves<T, DP>();
    const size_t lds = (size_t)NW * 2 * Tile<T, DP>::kBytes32;
    a.tiles = p.row_tiles32 * p.splits;
    const unsigned grid = attend_grid(&a);
    const hipError_t e = allow_lds<attend_step_kernel<T, DP, DMA>>(lds);
    if (e != hipSuccess) return e;
    attend_step_kernel<T, DP, DMA><<<grid, 64 * NW, lds, s>>>(a);
    if (p.splits > 1) {
      const int64_t rows = (int64_t)a.B * a.Hk * a.M;
      attend_join_kernel<T><<<(unsigned)((rows + 3) / 4), 256, 0, s>>>(a, p.row_tiles32);
    }
  } else {
    const size_t lds = (size_t)4 * fwd_keys<T, DP>() * C * 16;
    a.tiles = (int)((a.M + 127) / 128);
    const unsigned grid = attend_grid(&a);
    const hipError_t e = allow_lds<attend_fwd_kernel<T, DP, DMA>>(lds);
    if (e != hipSuccess) return e;
    attend_fwd_kernel<T, DP, DMA><<<grid, 256, lds, s>>>(a);
  }
  return hipGetLastError();
}

template <typename T>
static hipError_t attend_fwd_dp(const AttendPlan& p, const AttendArgs& a, hipStream_t s) {
  if (p.dma) {
    switch (p.DP) {
      case 32: return attend_fwd_t<T, 32, true>(p, a, s);
      case 64: return attend_fwd_t<T, 64, true>(p, a, s);
      case 96: return attend_fwd_t<T, 96, true>(p, a, s);
      case 128: return attend_fwd_t<T, 128, true>(p, a, s);
      case 192: return attend_fwd_t<T, 192, true>(p, a, s);
      default: return attend_fwd_t<T, 256, true>(p, a, s);
    }
  }
  // rows that go through registers: fewer sizes (64 pairs of four heads of 64,
  // 512 x 2048: 157 us, straight into LDS 91)
  return p.DP <= 64 ? attend_fwd_t<T, 64, false>(p, a, s)
         : p.DP <= 128 ? attend_fwd_t<T, 128, false>(p, a, s) : attend_fwd_t<T, 256, false>(p, a, s);
}

hipError_t launch_attend_fwd(const AttendPlan& p, const AttendArgs& a, hipStream_t s) {
  if (a.B == 0 || a.M == 0) return hipSuccess;
  Timed tm(8, s);
  if (p.dtype == LSTM_F32) return attend_fwd_dp<float>(p, a, s);
  if (p.dtype == LSTM_BF16) return attend_fwd_dp<bf16_t>(p, a, s);
  return attend_fwd_dp<f16_t>(p, a, s);
}

hipError_t launch_attend_bwd(const AttendPlan& p, const AttendArgs& a, hipStream_t s) {
  if (a.B == 0 || a.Hk == 0) return hipSuccess;
  Timed tm(8, s);
  if (p.dtype == LSTM_F32) return launch_attend_bwd_f32(p, a, s);
  if (p.dtype == LSTM_BF16) return launch_attend_bwd_bf16(p, a, s);
  return launch_attend_bwd_f16(p, a, s);
}

}  // namespace lstm
