// attend_bwd.hpp -- cross attention backward (gfx950): the kernels, which
// attend_bwd_f32.hip, _bf16.hip and _f16.hip each build for one storage type.
//
//   p = exp(s - lse), dp = dout . v, delta = dout . o, ds = scale p (dp - delta)
//   dq = sum_k ds k      dv = sum_rows p dout      dk = sum_rows ds q
//
// Two kernels, so that every sum stays in one wave's registers in a fixed
// order (no atomics): attend_dq_kernel walks over the keys with 32 query rows
// in registers, as the forward does, and writes delta on its way;
// attend_dkv_kernel walks over the query rows of every head of the group with
// 32 keys in registers.  Both recompute s and dp (seven products in place of
// five).  The matrix products are the bound, and beside them the reads of
// their fragments from LDS: 8 sequences, 32/8 heads of 128, 1024 x up to 4096
// keys, bf16: dq 470 us, 1090 TFLOP/s; dk and dv 750 us, 910 TFLOP/s.  At 64
// sequences, 16 heads of 64, 256 x 256 no unit is (dq 52 us, dk and dv 62;
// matrix units 15 and 18 % busy): the waves wait 40 % of their cycles for rows
// and barriers in loops of a few tiles.  In fp32, with few rows and keys (8
// sequences, 6/3 heads of 80, 37 x 191), dq takes 24 us and dk, dv 16, a chain
// of a few dependent tiles.
#pragma once
#include <type_traits>

#include "attend_common.hpp"

namespace lstm {

// The exponential gives 0 below 2^-126: p is carried 2^32 times larger through
// the products and their sums, in fp16, whose largest is 2^16, 2^15 times (p is
// an operand of dv, and its normal numbers then reach down to 2^-29 and not
// 2^-14), and the factor goes with `scale` when the sums are stored, so that
// the gradients of the smallest p survive as far as the type reaches.  In 16
// bits the factor is in the exponent, y + 32 or y + 15, whose rounding (2^-19
// of p) is far below the storage type's; in fp32 it would be the largest error
// of all, so there the factor is multiplied on, and the exponent of a small p
// is raised by 64 first.
template <typename T> constexpr float kCarry = std::is_same<T, f16_t>::value ? 32768.f : 4294967296.f;
template <typename T>
constexpr float kInExponent = std::is_same<T, float>::value ? 0.f : std::is_same<T, f16_t>::value ? 15.f : 32.f;
template <typename T>
__device__ __forceinline__ float exp_carried(float y) {
  if constexpr (std::is_same<T, float>::value) {
    const bool low = y < -64.f;
    return __builtin_amdgcn_exp2f(low ? y + 64.f : y) * (low ? kCarry<T> * 0x1p-64f : kCarry<T>);
  } else {
    return __builtin_amdgcn_exp2f(y);
  }
}

// Long sums in fp32 storage: after every kFoldTiles tiles the products' sums
// are added to a second set of registers and start again, so that a sum of n
// terms carries the rounding of about n / 16 + 16 tiles' additions and not of
// n (dq over 4096 keys: 1.1e-6 of its norm without).  In 16 bits the operands'
// rounding is far above it, and past 128 values a row there are no registers.
constexpr int kFoldTiles = 16;
template <typename T, int DP> constexpr bool kFold = std::is_same<T, float>::value && DP <= 128;
template <typename T, int DP>
struct Sums {
  static constexpr int N = kFold<T, DP> ? DP / 32 : 1;
  f32x16_t total[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) total[i] = zero16();
  }
  __device__ __forceinline__ void fold(f32x16_t* acc) {
    if constexpr (kFold<T, DP>) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        total[i] += acc[i];
        acc[i] = zero16();
      }
    }
  }
  __device__ __forceinline__ void finish(f32x16_t* acc) const {
    if constexpr (kFold<T, DP>) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += total[i];
    }
  }
};

// ds as an operand of fp16.  Its size is that of dout, which a scaled loss may
// bring to thousands, times p, which long keys bring to millionths: rounded as
// it stands, ds overflows or falls among the denormals although the gradients
// are normal numbers.  Each lane therefore carries the ds of its column (a row
// of dq, a key of dk) times a power of two `by`, which falls when a tile's
// largest passes 2^14 (to 2^9 .. 2^10, and the lane's sums with it) and else
// stays: what the reference of a softmax is to p.  It starts so high that
// nothing of 2^-66 or more stays below.  The other types have the exponents.
// (Backward without / with it, 16 sequences, 16/8 heads, 512 x 512, us: heads
// of 64 96 / 103, of 128 165 / 171, of 192 305 / 331, of 256 382 / 497; 8
// sequences, 32/8 heads of 128, 1024 x 4096: 1970 / 2053.)
template <typename T>
struct DsRange {
  static constexpr bool kMoves = std::is_same<T, f16_t>::value;
  float by = 0x1p80f;
  // N accumulators of 16 registers
  template <int N>
  __device__ __forceinline__ void fit(f32x16_t& ds, f32x16_t* acc) {
    if constexpr (kMoves) {
      float top = fabsf(ds[0]);
#pragma unroll
      for (int j = 1; j < 16; ++j) top = fmaxf(top, fabsf(ds[j]));
      top = fmaxf(top, other_half(top));
      const bool past = top * by > 0x1p14f;
      if (__ballot(past)) {
        const float to = past ? __builtin_ldexpf(1.f, 10 - __builtin_amdgcn_frexp_expf(top)) : by, r = to / by;
        by = to;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[i][j] *= r;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) ds[j] *= by;
    }
  }
  template <int N>
  __device__ __forceinline__ void finish(f32x16_t* acc) const {
    if constexpr (kMoves) {
      const float r = 1.f / by;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] *= r;
    }
  }
};

// What a query row (column lane % 32 of the products) keeps in registers.
template <typename T, int DP>
struct QueryRow {
  using TL = Tile<T, DP>;
  u32x4_t q[TL::KB], g[TL::KB];
  float lse2, delta;
  uint32_t t, h;
  bool ok;
  // r of the pair's M rows; `write`: its statistics go to memory for dk and dv
  __device__ __forceinline__ void load(const AttendArgs& a, int b, int hk, uint32_t r, bool write, int lane) {
    ok = r < a.M;
    t = r / a.G;
    h = hk * a.G + (r - t * a.G);
    load_row_frags<T, DP>((const T*)a.q + t * a.qs.t + b * a.qs.b + h * a.qs.h, a.D, a.whole & kWholeQ, ok, lane, q);
    load_row_frags<T, DP>((const T*)a.dout + t * a.gs.t + b * a.gs.b + h * a.gs.h, a.D, a.whole & kWholeG, ok, lane, g);
    // both operands a lane holds, and those of lane ^ 32
    const T* orow = (const T*)a.o + t * a.os.t + b * a.os.b + h * a.os.h;
    delta = 0.f;
#pragma unroll
    for (int kb = 0; kb < TL::KB; ++kb) {
      if (ok) {
        const u32x4_t ov = load_chunk<T>(orow, (2 * kb + (lane >> 5)) * vec_of<T>(), a.D, a.whole & kWholeO);
        float fo[vec_of<T>()], fg[vec_of<T>()];
        unpack<T>(ov, fo);
        unpack<T>(g[kb], fg);
#pragma unroll
        for (int j = 0; j < vec_of<T>(); ++j) delta += fo[j] * fg[j];
      }
    }
    delta += other_half(delta);
    lse2 = INFINITY;  // no row, or a row without keys: p = 0
    if (ok) {
      const int64_t li = ((int64_t)b * a.Hq + h) * a.Tq + t;
      const float v = a.lse[li];
      if (v != -INFINITY) lse2 = v * kLog2e - kInExponent<T>;
      if (write && lane < 32) *(float2*)(a.stats + 2 * li) = make_float2(lse2, delta);
    }
  }
  // adds 32 keys' terms to dq (the factor `scale` of ds goes to the end)
  __device__ __forceinline__ void tile(const char* kt, const char* vt, uint32_t bits, f32x16_t* dq, DsRange<T>& range,
                                       float c2, int lane) const {
    lane = tile_lane<DP == 256>(lane);
    f32x16_t s = zero16(), dp = zero16();
    constexpr int NDT = DP / 32;
    Ahead<2 * TL::KB, 8> rows;  // keys, then values
    Ahead<TL::PB * NDT, 4> cols;
    auto read_row = [&](int f) { return TL::row_frag(f < TL::KB ? kt : vt, 0, f % TL::KB, lane); };
    auto read_col = [&](int f) { return TL::col_frag(kt, TL::KR * (f / NDT), f % NDT, lane); };
    rows.start(read_row);
    rows.run(read_row, [&](int f, u32x4_t x) {
      if (f < TL::KB) s = Mm<T>::mac(x, q[f % TL::KB], s);
      else dp = Mm<T>::mac(x, g[f % TL::KB], dp);
    });
    cols.start(read_col);
    if (bits != 0xffffffffu) {
      const uint32_t mine = bits >> (4 * (lane >> 5));
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (!((mine >> reg_row(j, 0)) & 1)) s[j] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) s[j] = exp_carried<T>(__builtin_fmaf(s[j], c2, -lse2)) * (dp[j] - delta);
    range.template fit<NDT>(s, dq);
    u32x4_t ds[TL::PB];
#pragma unroll
    for (int pb = 0; pb < TL::PB; ++pb) ds[pb] = TL::reg_frag(s, pb);
    cols.run(read_col, [&](int f, u32x4_t x) { dq[f % NDT] = Mm<T>::mac(x, ds[f / NDT], dq[f % NDT]); });
  }
};

// Keys per tile: two double-buffered tiles in 64 KB where they can be two work-groups' share.
template <typename T, int DP> constexpr int dq_keys() { return 4 * 64 * Tile<T, DP>::C * 16 <= 64 * 1024 ? 64 : 32; }

template <typename T, int DP, bool DMA>
__global__ void __launch_bounds__(256, DP * sizeof(T) > 256 ? 1 : 2) attend_dq_kernel(AttendArgs a) {
  using TL = Tile<T, DP>;
  constexpr int NK = dq_keys<T, DP>(), TB = NK * TL::C * 16;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int grp, tile;
  if (!group_of(a, blockIdx.x, &grp, &tile)) return;
  const int b = grp / a.Hk, hk = grp - b * a.Hk;
  const int end = keys_of(a, b);
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_b : nullptr;
  QueryRow<T, DP> row;
  row.load(a, b, hk, (uint32_t)tile * 128 + w * 32 + (lane & 31), true, lane);
  Loader<T, DP, NK, 4, DMA> lk, lv;
  lk.init((const T*)a.k + b * a.ks.b + hk * a.ks.h, a.ks.t, a.D, a.whole & kWholeK, mask, w, lane);
  lv.init((const T*)a.v + b * a.vs.b + hk * a.vs.h, a.vs.t, a.D, a.whole & kWholeV, mask, w, lane);

  f32x16_t dq[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) dq[dt] = zero16();
  Sums<T, DP> sums;
  sums.clear();
  DsRange<T> range;
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
#pragma unroll
    for (int kt = 0; kt < NK / 32; ++kt)
      row.tile(cur + kt * TL::kBytes32, cur + TB + kt * TL::kBytes32, (uint32_t)(now >> (32 * kt)), dq, range, c2, lane);
    if (i % kFoldTiles == kFoldTiles - 1) sums.fold(dq);
  }
  sums.finish(dq);
  range.template finish<DP / 32>(dq);
  if (row.ok)
    store_col<T, DP>((T*)a.dq + row.t * a.dqs.t + b * a.dqs.b + row.h * a.dqs.h, dq, a.scale / kCarry<T>, a.D,
                     a.whole & kWholeDq, lane);
}

// Few rows: 32 per work-group, the tiles of keys dealt to its waves.
template <typename T, int DP, bool DMA>
__global__ void __launch_bounds__((64 * step_waves<T, DP>()), 1) attend_dq_few_kernel(AttendArgs a) {
  using TL = Tile<T, DP>;
  constexpr int NW = step_waves<T, DP>(), TB = TL::kBytes32;
  extern __shared__ __attribute__((aligned(16))) char lds[];  // per wave: K, V tile
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int grp, tile;
  if (!group_of(a, blockIdx.x, &grp, &tile)) return;
  const int b = grp / a.Hk, hk = grp - b * a.Hk;
  const int end = keys_of(a, b);
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_b : nullptr;
  Loader<T, DP, 32, 1, DMA> lk, lv;
  lk.init((const T*)a.k + b * a.ks.b + hk * a.ks.h, a.ks.t, a.D, a.whole & kWholeK, mask, 0, lane);
  lv.init((const T*)a.v + b * a.vs.b + hk * a.vs.h, a.vs.t, a.D, a.whole & kWholeV, mask, 0, lane);
  char* mine = lds + w * 2 * TB;
  const int n = (end + 31) / 32;
  uint64_t bits = 0;
  auto fetch = [&](int i) {
    lk.load(i * 32, end, mine);
    lv.load(i * 32, end, mine + TB);
    bits = key_bits(mask, i * 32, end, lane);
  };
  if (w < n) fetch(w);
  QueryRow<T, DP> row;
  row.load(a, b, hk, (uint32_t)tile * 32 + (lane & 31), w == 0, lane);
  f32x16_t dq[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) dq[dt] = zero16();
  DsRange<T> range;
  const float c2 = a.scale * kLog2e;
  for (int i = w; i < n; i += NW) {
    wait_vmem();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    row.tile(mine, mine + TB, (uint32_t)bits, dq, range, c2, lane);
    if (i + NW < n) {
      __builtin_amdgcn_s_waitcnt(kLgkm0);  // every fragment of this tile is read
      fetch(i + NW);
    }
  }
  range.template finish<DP / 32>(dq);
  T* out = (T*)a.dq + row.t * a.dqs.t + b * a.dqs.b + row.h * a.dqs.h;
  join_waves<T, DP>(dq, lds, a.D, w, lane, [&](int d, float v) {
    if (row.ok) out[d] = Elem<T>::from_f(as_f32(v * (a.scale / kCarry<T>)));
  });
}

// ---------------------------------------------------------------------------
// What 32 keys (column lane % 32) keep in registers.  DV, DK: which of the two
// gradients (both, where a wave has the registers).
template <typename T, int DP, bool DV, bool DK>
struct Keys {
  using TL = Tile<T, DP>;
  // Fragments read ahead.  16-bit rows of 128 values run two waves a SIMD in
  // 256 registers, 224 of them k, v, dk, dv, s and dp: there fewer are read
  // ahead, the columns' first ones only when s and dp have left their
  // registers, and the statistics a quarter at a time.  (A spilled register
  // in the loop costs more than its traffic: its reload waits for every
  // load into LDS before it.  Tried on 8 sequences, 32/8 heads of 128, 1024
  // x 4096: this 0.75 ms; with reloads 0.96; one wave a SIMD in 512 registers 1.11; 64 keys a
  // wave in 512, half the LDS reads, spilled, 2.0; dv and dk in two kernels
  // 0.43 + 0.53.)
  static constexpr bool kTight = sizeof(T) == 2 && DP == 128;
  static constexpr int kAheadRows = kTight ? 4 : 8, kAheadGrads = kTight ? 2 : 8, kAheadCols = 4;
  u32x4_t k[TL::KB], v[DK ? TL::KB : 1];
  f32x16_t dk[DK ? DP / 32 : 1], dv[DV ? DP / 32 : 1];
  Sums<T, DP> sk, sv;
  DsRange<T> range;
  __device__ __forceinline__ void fold() {
    if constexpr (DK) sk.fold(dk);
    if constexpr (DV) sv.fold(dv);
  }
  __device__ __forceinline__ void finish() {
    if constexpr (DK) {
      sk.finish(dk);
      range.template finish<DP / 32>(dk);
    }
    if constexpr (DV) sv.finish(dv);
  }
  __device__ __forceinline__ void clear() {
    sk.clear();
    sv.clear();
#pragma unroll
    for (int dt = 0; dt < (DK ? DP / 32 : 1); ++dt) dk[dt] = zero16();
#pragma unroll
    for (int dt = 0; dt < (DV ? DP / 32 : 1); ++dt) dv[dt] = zero16();
  }
  __device__ __forceinline__ void load(const AttendArgs& a, int b, int hk, int key, bool ok, int lane) {
    load_row_frags<T, DP>((const T*)a.k + key * a.ks.t + b * a.ks.b + hk * a.ks.h, a.D, a.whole & kWholeK, ok, lane, k);
    if constexpr (DK)
      load_row_frags<T, DP>((const T*)a.v + key * a.vs.t + b * a.vs.b + hk * a.vs.h, a.D, a.whole & kWholeV, ok, lane,
                            v);
  }
  // adds the terms of 32 query rows: their q and dout tiles and (lse2, delta)
  // pairs.  Rows past the last have zeros in all of them and add nothing.
  __device__ __forceinline__ void tile(const char* qt, const char* gt, const float* stat, float c2, int lane) {
    lane = tile_lane<kTight || DP == 256 || (sizeof(T) == 4 && (DP == 64 || DP == 128))>(lane);
    f32x16_t s = zero16(), dp = zero16();
    constexpr int NDT = DP / 32, NG = (DV ? 1 : 0) + (DK ? 1 : 0);
    Ahead<TL::KB, kAheadRows> rq;
    Ahead<TL::KB, kAheadGrads> rg;
    Ahead<TL::PB * NDT * NG, kAheadCols> cols;  // k-block, d-tile, dout then q
    auto read_q = [&](int f) { return TL::row_frag(qt, 0, f, lane); };
    auto read_g = [&](int f) { return TL::row_frag(gt, 0, f, lane); };
    auto read_col = [&](int f) {
      return TL::col_frag(DV && f % NG == 0 ? gt : qt, TL::KR * (f / NG / NDT), f / NG % NDT, lane);
    };
    rq.start(read_q);
    rq.run(read_q, [&](int f, u32x4_t x) { s = Mm<T>::mac(x, k[f], s); });
    if constexpr (DK) {
      rg.start(read_g);
      rg.run(read_g, [&](int f, u32x4_t x) { dp = Mm<T>::mac(x, v[f], dp); });
    }
    if constexpr (!kTight) cols.start(read_col);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* at = stat + 2 * reg_row(4 * j, lane);
      const f32x4_t x = *(const f32x4_t*)at, y = *(const f32x4_t*)(at + 4);
      const float L[4] = {x[0], x[2], y[0], y[2]}, d[4] = {x[1], x[3], y[1], y[3]};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[4 * j + e] = exp_carried<T>(__builtin_fmaf(s[4 * j + e], c2, -L[e]));
        if constexpr (DK) dp[4 * j + e] = s[4 * j + e] * (dp[4 * j + e] - d[e]);
      }
      if constexpr (kTight) __builtin_amdgcn_sched_barrier(0);
    }
    u32x4_t p[TL::PB], ds[TL::PB];
    if constexpr (DV)
#pragma unroll
      for (int pb = 0; pb < TL::PB; ++pb) p[pb] = TL::reg_frag(s, pb);
    if constexpr (DK) {
      range.template fit<NDT>(dp, dk);
#pragma unroll
      for (int pb = 0; pb < TL::PB; ++pb) ds[pb] = TL::reg_frag(dp, pb);
    }
    if constexpr (kTight) {
      __builtin_amdgcn_sched_barrier(0);
      cols.start(read_col);
    }
    cols.run(read_col, [&](int f, u32x4_t x) {
      const int pb = f / NG / NDT, dt = f / NG % NDT;
      if (DV && f % NG == 0) dv[DV ? dt : 0] = Mm<T>::mac(x, p[pb], dv[DV ? dt : 0]);
      else dk[DK ? dt : 0] = Mm<T>::mac(x, ds[pb], dk[DK ? dt : 0]);
    });
  }
};

// Tiles of NR query rows of the heads that share a key head: tile i is rows
// [NR (i % nt), +NR) of head i / nt.  A stage in LDS: the q tile, the dout
// tile, and for each wave its own copy of the rows' (lse2, delta) pairs.
template <typename T, int DP, int NR, int NW, bool DMA>
struct QueryTiles {
  using TL = Tile<T, DP>;
  using Load = Loader<T, DP, NR, NW, DMA>;
  static constexpr int kTile = NR / 32 * TL::kBytes32, kStat = NR * 8, kStage = 2 * kTile + NW * kStat;
  static constexpr int kStatLoads = NR / 32;
  // every wave has as many loads, and two stages' can be told apart
  static constexpr bool kCounted = DMA && Load::kTotal % NW == 0 && 2 * (2 * Load::kLoads + kStatLoads) <= 63;
  static constexpr int kLoads = 2 * Load::kLoads + kStatLoads;     // of a stage and wave
  Load lq, lg;
  const float* st0;  // of this head's rows
  int nt, n, Tq, w, lane;
  int64_t qh, gh;
  int t0;  // first row of the tile that fetch() loads
  __device__ __forceinline__ void init(const AttendArgs& a, int b, int hk, int w_, int lane_) {
    w = w_; lane = lane_;
    Tq = a.Tq; qh = a.qs.h; gh = a.gs.h;
    lq.init((const T*)a.q + b * a.qs.b + (int64_t)hk * a.G * qh, a.qs.t, a.D, a.whole & kWholeQ, nullptr, w, lane);
    lg.init((const T*)a.dout + b * a.gs.b + (int64_t)hk * a.G * gh, a.gs.t, a.D, a.whole & kWholeG, nullptr, w, lane);
    st0 = a.stats + 2 * ((int64_t)b * a.Hq + (int64_t)hk * a.G) * Tq;
    nt = (Tq + NR - 1) / NR;
    n = nt * a.G;
    t0 = 0;
  }
  // on by `by` tiles
  __device__ __forceinline__ void skip(int by) {
    t0 += NR * by;
    while (t0 >= NR * nt && nt > 0) {
      t0 -= NR * nt;
      lq.p += qh;
      lg.p += gh;
      st0 += 2 * (int64_t)Tq;
    }
  }
  __device__ __forceinline__ static const float* stat(const char* stage, int w) {
    return (const float*)(stage + 2 * kTile + w * kStat);
  }
  __device__ __forceinline__ void fetch(char* stage) {
    lq.load(t0, Tq, stage);
    lg.load(t0, Tq, stage + kTile);
    const float* s = st0 + 2 * (int64_t)t0;
    const int rows = Tq - t0 < NR ? Tq - t0 : NR;
    char* to = stage + 2 * kTile + w * kStat;
    if constexpr (DMA) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)s, 0, rows * 8, 0x00020000);
#pragma unroll
      for (int i = 0; i < kStatLoads; ++i) lds_dma4(r, to + 256 * i, 256 * i + lane * 4);
    } else {
      for (int i = lane; i < 2 * NR; i += 64) ((float*)to)[i] = i < 2 * rows ? s[i] : 0.f;
    }
  }
};

// 128 keys per work-group, 32 per wave, which share the tiles of query rows,
// in a ring of stages (one barrier a tile: the stage that is loaded next was
// read before it): 64 rows a stage and two stages up to rows of 128 bytes
// (64 sequences, 16 heads of 64, 256 x 256: 62 us, with stages of 32 rows
// 66-69), else 32 rows and as many stages, up to four, as leave LDS to two
// work-groups.
template <typename T, int DP> constexpr int dkv_rows() { return DP * sizeof(T) <= 128 ? 64 : 32; }
template <typename T, int DP, bool DMA> constexpr int dkv_ring() {
  constexpr int stage = QueryTiles<T, DP, dkv_rows<T, DP>(), 4, DMA>::kStage;
  return dkv_rows<T, DP>() == 64 ? 2 : 4 * stage <= 96 * 1024 ? 4 : 3 * stage <= 150 * 1024 ? 3 : 2;
}

template <typename T, int DP, bool DMA, bool DV, bool DK>
__global__ void __launch_bounds__(256, DP * sizeof(T) > 256 ? 1 : 2) attend_dkv_kernel(AttendArgs a) {
  constexpr int TB = Tile<T, DP>::kBytes32, R = dkv_ring<T, DP, DMA>();
  using Tiles = QueryTiles<T, DP, dkv_rows<T, DP>(), 4, DMA>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int grp, tile;
  if (!group_of(a, blockIdx.x, &grp, &tile)) return;
  const int b = grp / a.Hk, hk = grp - b * a.Hk;
  const int end = keys_of(a, b);
  const int key = tile * 128 + w * 32 + (lane & 31);
  // whether key takes part, asked again at the end: kept, it would take registers from the loop
  auto takes_part = [&] { return key < end && (!a.mask || a.mask[b * a.mask_b + key] != 0); };
  Keys<T, DP, DV, DK> me;
  me.clear();
  if (tile * 128 < end) {
    const float c2 = a.scale * kLog2e;
    Tiles qt;
    qt.init(a, b, hk, w, lane);
    me.load(a, b, hk, key, takes_part(), lane);
    wait_vmem();  // from here on the ring's loads alone are counted
#pragma unroll
    for (int i = 0; i < R - 1; ++i)
      if (i < qt.n) {
        qt.fetch(lds + i * Tiles::kStage);
        qt.skip(1);
      }
    int at = 0;  // stage of tile i
    for (int i = 0; i < qt.n; ++i) {
      // tile i has arrived; up to R - 2 younger ones may be on their way
      const int young = qt.n - 1 - i;
      if (Tiles::kCounted && R == 4 && young >= 2) __builtin_amdgcn_s_waitcnt(vmcnt_imm(Tiles::kCounted ? 2 * Tiles::kLoads : 0));
      else if (Tiles::kCounted && R >= 3 && young >= 1) __builtin_amdgcn_s_waitcnt(vmcnt_imm(Tiles::kCounted ? Tiles::kLoads : 0));
      else wait_vmem();
      __syncthreads();
      char* cur = lds + at * Tiles::kStage;
      if (i + R - 1 < qt.n) {
        qt.fetch(lds + ((at + R - 1) % R) * Tiles::kStage);
        qt.skip(1);
      }
#pragma unroll
      for (int h = 0; h < Tiles::kStatLoads; ++h)
        me.tile(cur + h * TB, cur + Tiles::kTile + h * TB, Tiles::stat(cur, w) + 64 * h, c2, lane);
      if (i % kFoldTiles == kFoldTiles - 1) me.fold();
      at = (at + 1) % R;
    }
    me.finish();
  }
  if (key >= a.Tk) return;
  const bool ok = takes_part();  // keys of no query: zeros, whatever the products of their zeroed rows were
  if constexpr (DK)
    store_col<T, DP>((T*)a.dk + key * a.dks.t + b * a.dks.b + hk * a.dks.h, me.dk, a.scale / kCarry<T>, a.D,
                     a.whole & kWholeDk, lane, ok);
  if constexpr (DV)
    store_col<T, DP>((T*)a.dv + key * a.dvs.t + b * a.dvs.b + hk * a.dvs.h, me.dv, 1.f / kCarry<T>, a.D,
                     a.whole & kWholeDv, lane, ok);
}

// Few keys: 32 per work-group, the tiles of query rows dealt to its waves.
template <typename T, int DP, bool DMA, bool DV, bool DK>
__global__ void __launch_bounds__((64 * step_waves<T, DP>()), 1) attend_dkv_few_kernel(AttendArgs a) {
  constexpr int NW = step_waves<T, DP>(), TB = Tile<T, DP>::kBytes32;
  using Tiles = QueryTiles<T, DP, 32, 1, DMA>;
  extern __shared__ __attribute__((aligned(16))) char lds[];  // per wave: a stage
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int grp, tile;
  if (!group_of(a, blockIdx.x, &grp, &tile)) return;
  const int b = grp / a.Hk, hk = grp - b * a.Hk;
  const int end = keys_of(a, b);
  const int key = tile * 32 + (lane & 31);
  const bool ok = key < end && (!a.mask || a.mask[b * a.mask_b + key] != 0);
  char* mine = lds + w * Tiles::kStage;
  Keys<T, DP, DV, DK> me;
  me.clear();
  if (tile * 32 < end) {
    const float c2 = a.scale * kLog2e;
    Tiles qt;
    qt.init(a, b, hk, 0, lane);
    qt.skip(w);
    if (w < qt.n) qt.fetch(mine);
    me.load(a, b, hk, key, ok, lane);
    for (int i = w; i < qt.n; i += NW) {
      wait_vmem();
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      me.tile(mine, mine + TB, Tiles::stat(mine, 0), c2, lane);
      if (i + NW < qt.n) {
        __builtin_amdgcn_s_waitcnt(kLgkm0);  // every fragment of this tile is read
        qt.skip(NW);
        qt.fetch(mine);
      }
    }
  }
  const bool store = key < a.Tk;
  if constexpr (DK) {
    me.range.template finish<DP / 32>(me.dk);
    T* out = (T*)a.dk + key * a.dks.t + b * a.dks.b + hk * a.dks.h;
    join_waves<T, DP>(me.dk, lds, a.D, w, lane, [&](int d, float v) {
      if (store) out[d] = Elem<T>::from_f(ok ? as_f32(v * (a.scale / kCarry<T>)) : 0.f);
    });
  }
  if constexpr (DV) {
    T* out = (T*)a.dv + key * a.dvs.t + b * a.dvs.b + hk * a.dvs.h;
    join_waves<T, DP>(me.dv, lds, a.D, w, lane, [&](int d, float v) {
      if (store) out[d] = Elem<T>::from_f(ok ? as_f32(v / kCarry<T>) : 0.f);
    });
  }
}

// ---------------------------------------------------------------------------
template <typename T, int DP, bool DMA, bool DV, bool DK>
static hipError_t attend_dkv_t(const AttendPlan& p, AttendArgs a, hipStream_t s) {
  const bool few = p.few_keys;
  const size_t lds = few ? step_waves<T, DP>() * (size_t)QueryTiles<T, DP, 32, 1, DMA>::kStage
                         : dkv_ring<T, DP, DMA>() * (size_t)QueryTiles<T, DP, dkv_rows<T, DP>(), 4, DMA>::kStage;
  a.tiles = few ? (a.Tk + 31) / 32 : (a.Tk + 127) / 128;
  const unsigned grid = attend_grid(&a);
  const hipError_t e = few ? allow_lds<attend_dkv_few_kernel<T, DP, DMA, DV, DK>>(lds)
                           : allow_lds<attend_dkv_kernel<T, DP, DMA, DV, DK>>(lds);
  if (e != hipSuccess) return e;
  if (few)
    attend_dkv_few_kernel<T, DP, DMA, DV, DK><<<grid, 64 * step_waves<T, DP>(), lds, s>>>(a);
  else
    attend_dkv_kernel<T, DP, DMA, DV, DK><<<grid, 256, lds, s>>>(a);
  return hipGetLastError();
}

template <typename T, int DP, bool DMA>
static hipError_t attend_bwd_t(const AttendPlan& p, const AttendArgs& a0, hipStream_t s) {
  AttendArgs a = a0;
  if (a.M > 0) {
    const bool few = p.few_rows;
    const size_t lds = few ? (size_t)2 * step_waves<T, DP>() * Tile<T, DP>::kBytes32
                           : (size_t)4 * dq_keys<T, DP>() * Tile<T, DP>::C * 16;
    a.tiles = few ? p.row_tiles32 : (int)((a.M + 127) / 128);
    const unsigned grid = attend_grid(&a);
    const hipError_t e =
        few ? allow_lds<attend_dq_few_kernel<T, DP, DMA>>(lds) : allow_lds<attend_dq_kernel<T, DP, DMA>>(lds);
    if (e != hipSuccess) return e;
    if (few)
      attend_dq_few_kernel<T, DP, DMA><<<grid, 64 * step_waves<T, DP>(), lds, s>>>(a);
    else
      attend_dq_kernel<T, DP, DMA><<<grid, 256, lds, s>>>(a);
  }
  if (a.Tk > 0) {
    // fp32 rows of more than 128 values leave no registers for both sums, nor
    // do fp16 rows of 256 beside the moving range (16 sequences, 16/8 heads,
    // 512 x 512, the whole backward: one launch 924 us, spilled, two 497)
    if constexpr (DP * sizeof(T) > 512 || (DsRange<T>::kMoves && DP == 256)) {
      const hipError_t e = attend_dkv_t<T, DP, DMA, true, false>(p, a, s);
      if (e != hipSuccess) return e;
      return attend_dkv_t<T, DP, DMA, false, true>(p, a, s);
    } else {
      return attend_dkv_t<T, DP, DMA, true, true>(p, a, s);
    }
  }
  return hipGetLastError();
}

template <typename T>
static hipError_t attend_bwd_dp(const AttendPlan& p, const AttendArgs& a, hipStream_t s) {
  if (p.dma) {
    switch (p.DP) {
      case 32: return attend_bwd_t<T, 32, true>(p, a, s);
      case 64: return attend_bwd_t<T, 64, true>(p, a, s);
      case 96: return attend_bwd_t<T, 96, true>(p, a, s);
      case 128: return attend_bwd_t<T, 128, true>(p, a, s);
      case 192: return attend_bwd_t<T, 192, true>(p, a, s);
      default: return attend_bwd_t<T, 256, true>(p, a, s);
    }
  }
  return p.DP <= 64 ? attend_bwd_t<T, 64, false>(p, a, s)
         : p.DP <= 128 ? attend_bwd_t<T, 128, false>(p, a, s) : attend_bwd_t<T, 256, false>(p, a, s);
}

}  // namespace lstm
