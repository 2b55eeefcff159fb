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
// 32 keys in registers.  Both recompute s (seven products in place of five).
#pragma once
#include <type_traits>

#include "attend_common.hpp"

namespace lstm {

// The exponential gives 0 below 2^-126: where the storage type has the range,
// p is carried 2^32 times larger through the products and their sums, and the
// factor goes with `scale` when the sums are stored, so that the gradients of
// the smallest p survive as far as the type reaches.  (fp16 would overflow.)
// In bf16 the factor is in the exponent, y + 32, whose rounding (2^-19 of p)
// is far below the storage type's; in fp32 it would be the largest error of
// all, so there the factor is multiplied on, and the exponent of a small p is
// raised by 64 first.
template <typename T> constexpr float kCarry = std::is_same<T, f16_t>::value ? 1.f : 4294967296.f;
template <typename T> constexpr float kInExponent = std::is_same<T, bf16_t>::value ? 32.f : 0.f;
template <typename T>
__device__ __forceinline__ float exp_carried(float y) {
  if constexpr (std::is_same<T, float>::value) {
    const bool low = y < -64.f;
    return __builtin_amdgcn_exp2f(low ? y + 64.f : y) * (low ? kCarry<T> * 0x1p-64f : kCarry<T>);
  } else {
    return __builtin_amdgcn_exp2f(y);
  }
}

// What a query row (column lane % 32 of the products) keeps in registers.
template <typename T, int DP>
struct QueryRow {
  using TL = Tile<T, DP>;
  u32x4_t q[TL::KB], g[TL::KB];
  float lse2, delta;
  uint32_t t, h;
  bool ok;
  // r of the pair's M rows; also writes its delta
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
      if (write && lane < 32) a.delta[li] = delta;
    }
  }
  // adds 32 keys' terms to dq (the factor `scale` of ds goes to the end)
  __device__ __forceinline__ void tile(const char* kt, const char* vt, uint32_t bits, f32x16_t* dq, float c2,
                                       int lane) const {
    f32x16_t s = zero16(), dp = zero16();
#pragma unroll
    for (int kb = 0; kb < TL::KB; ++kb) s = Mm<T>::mac(TL::row_frag(kt, 0, kb, lane), q[kb], s);
#pragma unroll
    for (int kb = 0; kb < TL::KB; ++kb) dp = Mm<T>::mac(TL::row_frag(vt, 0, kb, lane), g[kb], dp);
    if (bits != 0xffffffffu) {
      const uint32_t mine = bits >> (4 * (lane >> 5));
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (!((mine >> reg_row(j, 0)) & 1)) s[j] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) s[j] = exp_carried<T>(__builtin_fmaf(s[j], c2, -lse2)) * (dp[j] - delta);
#pragma unroll
    for (int pb = 0; pb < TL::PB; ++pb) {
      const u32x4_t ds = TL::reg_frag(s, pb);
#pragma unroll
      for (int dt = 0; dt < DP / 32; ++dt) dq[dt] = Mm<T>::mac(TL::col_frag(kt, TL::KR * pb, dt, lane), ds, dq[dt]);
    }
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
      row.tile(cur + kt * TL::kBytes32, cur + TB + kt * TL::kBytes32, (uint32_t)(now >> (32 * kt)), dq, c2, lane);
  }
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
  const float c2 = a.scale * kLog2e;
  for (int i = w; i < n; i += NW) {
    wait_vmem();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    row.tile(mine, mine + TB, (uint32_t)bits, dq, c2, lane);
    if (i + NW < n) {
      __builtin_amdgcn_s_waitcnt(kLgkm0);  // every fragment of this tile is read
      fetch(i + NW);
    }
  }
  T* out = (T*)a.dq + row.t * a.dqs.t + b * a.dqs.b + row.h * a.dqs.h;
  join_waves<T, DP>(dq, lds, a.D, w, lane, [&](int d, float v) {
    if (row.ok) out[d] = Elem<T>::from_f(as_f32(v * (a.scale / kCarry<T>)));
  });
}

// ---------------------------------------------------------------------------
// What a key (column lane % 32) keeps in registers.  DV, DK: which of the two
// gradients (both, where a wave has the registers).
template <typename T, int DP, bool DV, bool DK>
struct Key {
  using TL = Tile<T, DP>;
  u32x4_t k[TL::KB], v[DK ? TL::KB : 1];
  f32x16_t dk[DK ? DP / 32 : 1], dv[DV ? DP / 32 : 1];
  __device__ __forceinline__ void clear() {
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
  // adds the terms of 32 query rows: their q and dout tiles, lse2[32] and
  // delta[32] behind it
  __device__ __forceinline__ void tile(const char* qt, const char* gt, const float* stat, float c2, int lane) {
    f32x16_t s = zero16(), dp = zero16();
#pragma unroll
    for (int kb = 0; kb < TL::KB; ++kb) s = Mm<T>::mac(TL::row_frag(qt, 0, kb, lane), k[kb], s);
    if constexpr (DK) {
#pragma unroll
      for (int kb = 0; kb < TL::KB; ++kb) dp = Mm<T>::mac(TL::row_frag(gt, 0, kb, lane), v[kb], dp);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x4_t L = *(const f32x4_t*)(stat + reg_row(4 * j, lane));
#pragma unroll
      for (int e = 0; e < 4; ++e) s[4 * j + e] = exp_carried<T>(__builtin_fmaf(s[4 * j + e], c2, -L[e]));
    }
    if constexpr (DV) {
#pragma unroll
      for (int pb = 0; pb < TL::PB; ++pb) {
        const u32x4_t p = TL::reg_frag(s, pb);
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) dv[dt] = Mm<T>::mac(TL::col_frag(gt, TL::KR * pb, dt, lane), p, dv[dt]);
      }
    }
    if constexpr (DK) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4_t d = *(const f32x4_t*)(stat + 32 + reg_row(4 * j, lane));
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * j + e] *= dp[4 * j + e] - d[e];
      }
#pragma unroll
      for (int pb = 0; pb < TL::PB; ++pb) {
        const u32x4_t ds = TL::reg_frag(s, pb);
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) dk[dt] = Mm<T>::mac(TL::col_frag(qt, TL::KR * pb, dt, lane), ds, dk[dt]);
      }
    }
  }
};

// Tiles of 32 query rows of the heads that share a key head: tile i is rows
// [32 (i % nt), +32) of head i / nt.
template <typename T, int DP, int NW, bool DMA>
struct QueryTiles {
  using TL = Tile<T, DP>;
  Loader<T, DP, 32, NW, DMA> lq, lg;
  const T *q0, *g0;
  int64_t row0;  // of lse and delta
  int nt, n;
  float l, d;    // of this lane's row (lanes 0 .. 31)
  __device__ __forceinline__ void init(const AttendArgs& a, int b, int hk, int w, int lane) {
    q0 = (const T*)a.q + b * a.qs.b + (int64_t)hk * a.G * a.qs.h;
    g0 = (const T*)a.dout + b * a.gs.b + (int64_t)hk * a.G * a.gs.h;
    lq.init(q0, a.qs.t, a.D, a.whole & kWholeQ, nullptr, w, lane);
    lg.init(g0, a.gs.t, a.D, a.whole & kWholeG, nullptr, w, lane);
    row0 = ((int64_t)b * a.Hq + (int64_t)hk * a.G) * a.Tq;
    nt = (a.Tq + 31) / 32;
    n = nt * a.G;
  }
  __device__ __forceinline__ void fetch(const AttendArgs& a, int i, char* lds, bool stats, int lane) {
    const int hd = i / nt, t0 = (i - hd * nt) * 32;
    lq.p = q0 + hd * a.qs.h;
    lg.p = g0 + hd * a.gs.h;
    lq.load(t0, a.Tq, lds);
    lg.load(t0, a.Tq, lds + TL::kBytes32);
    l = INFINITY;  // rows past the last, and rows without keys: p = 0
    d = 0.f;
    const int t = t0 + lane;
    if (stats && lane < 32 && t < a.Tq) {
      const int64_t li = row0 + (int64_t)hd * a.Tq + t;
      const float x = a.lse[li];
      if (x != -INFINITY) l = x * kLog2e - kInExponent<T>;
      d = a.delta[li];
    }
  }
  __device__ __forceinline__ void keep(float* stat, bool stats, int lane) const {
    if (stats && lane < 32) {
      stat[lane] = l;
      stat[32 + lane] = d;
    }
  }
};

// 128 keys per work-group, 32 per wave, which share the tiles of query rows.
template <typename T, int DP, bool DMA, bool DV, bool DK>
__global__ void __launch_bounds__(256, DP * sizeof(T) > 256 ? 1 : 2) attend_dkv_kernel(AttendArgs a) {
  constexpr int TB = Tile<T, DP>::kBytes32;
  extern __shared__ __attribute__((aligned(16))) char lds[];  // q, dout tiles, twice
  __shared__ __attribute__((aligned(16))) float stat[2][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int grp, tile;
  if (!group_of(a, blockIdx.x, &grp, &tile)) return;
  const int b = grp / a.Hk, hk = grp - b * a.Hk;
  const int end = keys_of(a, b);
  const int key = tile * 128 + w * 32 + (lane & 31);
  const bool ok = key < end && (!a.mask || a.mask[b * a.mask_b + key] != 0);
  Key<T, DP, DV, DK> me;
  me.clear();
  if (tile * 128 < end) {
    me.load(a, b, hk, key, ok, lane);
    const float c2 = a.scale * kLog2e;
    QueryTiles<T, DP, 4, DMA> qt;
    qt.init(a, b, hk, w, lane);
    if (qt.n > 0) {
      qt.fetch(a, 0, lds, w == 0, lane);
      qt.keep(stat[0], w == 0, lane);
    }
    for (int i = 0; i < qt.n; ++i) {
      wait_vmem();
      __syncthreads();
      const int buf = i & 1;
      const char* cur = lds + buf * 2 * TB;
      if (i + 1 < qt.n) qt.fetch(a, i + 1, lds + (buf ^ 1) * 2 * TB, w == 0, lane);
      me.tile(cur, cur + TB, stat[buf], c2, lane);
      if (i + 1 < qt.n) qt.keep(stat[buf ^ 1], w == 0, lane);
    }
  }
  if (key >= a.Tk) return;
  if (!ok) me.clear();  // keys of no query: zeros, whatever the products of their zeroed rows were
  if constexpr (DK)
    store_col<T, DP>((T*)a.dk + key * a.dks.t + b * a.dks.b + hk * a.dks.h, me.dk, a.scale / kCarry<T>, a.D,
                     a.whole & kWholeDk, lane);
  if constexpr (DV)
    store_col<T, DP>((T*)a.dv + key * a.dvs.t + b * a.dvs.b + hk * a.dvs.h, me.dv, 1.f / kCarry<T>, a.D,
                     a.whole & kWholeDv, lane);
}

// Few keys: 32 per work-group, the tiles of query rows dealt to its waves.
template <typename T, int DP, bool DMA, bool DV, bool DK>
__global__ void __launch_bounds__((64 * step_waves<T, DP>()), 1) attend_dkv_few_kernel(AttendArgs a) {
  constexpr int NW = step_waves<T, DP>(), TB = Tile<T, DP>::kBytes32;
  extern __shared__ __attribute__((aligned(16))) char lds[];  // per wave: q, dout tile
  __shared__ __attribute__((aligned(16))) float stat[NW][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int grp, tile;
  if (!group_of(a, blockIdx.x, &grp, &tile)) return;
  const int b = grp / a.Hk, hk = grp - b * a.Hk;
  const int end = keys_of(a, b);
  const int key = tile * 32 + (lane & 31);
  const bool ok = key < end && (!a.mask || a.mask[b * a.mask_b + key] != 0);
  char* mine = lds + w * 2 * TB;
  Key<T, DP, DV, DK> me;
  me.clear();
  if (tile * 32 < end) {
    const float c2 = a.scale * kLog2e;
    QueryTiles<T, DP, 1, DMA> qt;
    qt.init(a, b, hk, 0, lane);
    if (w < qt.n) qt.fetch(a, w, mine, true, lane);
    me.load(a, b, hk, key, ok, lane);
    for (int i = w; i < qt.n; i += NW) {
      qt.keep(stat[w], true, lane);
      wait_vmem();
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      me.tile(mine, mine + TB, stat[w], c2, lane);
      if (i + NW < qt.n) {
        __builtin_amdgcn_s_waitcnt(kLgkm0);  // every fragment of this tile is read
        qt.fetch(a, i + NW, mine, true, lane);
      }
    }
  }
  const bool store = key < a.Tk;
  if constexpr (DK) {
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
  const size_t lds = (few ? 2 * step_waves<T, DP>() : 4) * (size_t)Tile<T, DP>::kBytes32;
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
    // fp32 rows of more than 128 values leave no registers for both sums
    if constexpr (DP * sizeof(T) > 512) {
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
