// attend_bwd.hip -- cross attention backward (gfx950).
//
//   p = exp(s - lse), dp = dout . v, delta = dout . o, ds = scale p (dp - delta)
//   dq = sum_k ds k      dv = sum_rows p dout      dk = sum_rows ds q
//
// Two kernels, so that every sum stays in one wave's registers in a fixed
// order (no atomics): attend_dq_kernel walks over the keys with 32 query rows
// in registers, as the forward does, and writes delta on its way;
// attend_dkv_kernel walks over the query rows of every head of the group with
// 32 keys in registers.  Both recompute s (seven products in place of five).
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
  const uint32_t r = (uint32_t)tile * 128 + w * 32 + (lane & 31);
  const bool ok = r < a.M;
  const uint32_t t = r / a.G, h = hk * a.G + (r - t * a.G);

  u32x4_t q[TL::KB], g[TL::KB];
  const T* grow = (const T*)a.dout + t * a.gs.t + b * a.gs.b + h * a.gs.h;
  load_row_frags<T, DP>((const T*)a.q + t * a.qs.t + b * a.qs.b + h * a.qs.h, a.D, a.whole & kWholeQ, ok, lane, q);
  load_row_frags<T, DP>(grow, a.D, a.whole & kWholeG, ok, lane, g);
  // delta: both operands a lane holds, and those of lane ^ 32
  float delta = 0.f;
  {
    const T* orow = (const T*)a.o + t * a.os.t + b * a.os.b + h * a.os.h;
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
  }
  const int64_t li = ((int64_t)b * a.Hq + h) * a.Tq + t;
  float lse2 = INFINITY;  // no row, or a row without keys: p = 0
  if (ok) {
    const float v = a.lse[li];
    if (v != -INFINITY) lse2 = v * kLog2e - kInExponent<T>;
    if (lane < 32) a.delta[li] = delta;
  }
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
    for (int kt = 0; kt < NK / 32; ++kt) {
      f32x16_t s = zero16(), dp = zero16();
#pragma unroll
      for (int kb = 0; kb < TL::KB; ++kb) s = Mm<T>::mac(TL::row_frag(cur, 32 * kt, kb, lane), q[kb], s);
#pragma unroll
      for (int kb = 0; kb < TL::KB; ++kb) dp = Mm<T>::mac(TL::row_frag(cur + TB, 32 * kt, kb, lane), g[kb], dp);
      const uint32_t mine = (uint32_t)(now >> (32 * kt));
      if (mine != 0xffffffffu) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (!((mine >> reg_row(j, lane)) & 1)) s[j] = -INFINITY;
      }
      // the factor `scale` of ds goes to the end
#pragma unroll
      for (int j = 0; j < 16; ++j)
        s[j] = exp_carried<T>(__builtin_fmaf(s[j], c2, -lse2)) * (dp[j] - delta);
#pragma unroll
      for (int pb = 0; pb < TL::PB; ++pb) {
        const u32x4_t ds = TL::reg_frag(s, pb);
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
          dq[dt] = Mm<T>::mac(TL::col_frag(cur, 32 * kt + TL::KR * pb, dt, lane), ds, dq[dt]);
      }
    }
  }
  if (ok)
    store_col<T, DP>((T*)a.dq + t * a.dqs.t + b * a.dqs.b + h * a.dqs.h, dq, a.scale / kCarry<T>, a.D, a.whole & kWholeDq, lane);
}

// ---------------------------------------------------------------------------
// 128 keys per work-group, 32 per wave; tiles of 32 query rows of one head.
// DV, DK: which of the two it computes (both, where a wave has the registers).
template <typename T, int DP, bool DMA, bool DV, bool DK>
__global__ void __launch_bounds__(256, DP * sizeof(T) > 256 ? 1 : 2) attend_dkv_kernel(AttendArgs a) {
  using TL = Tile<T, DP>;
  constexpr int NR = 32, TB = NR * TL::C * 16;
  extern __shared__ __attribute__((aligned(16))) char lds[];  // q, dout tiles, twice
  __shared__ __attribute__((aligned(16))) float stat[2][2][NR];  // lse2, delta
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int grp, tile;
  if (!group_of(a, blockIdx.x, &grp, &tile)) return;
  const int b = grp / a.Hk, hk = grp - b * a.Hk;
  const int end = keys_of(a, b);
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_b : nullptr;
  const int key = tile * 128 + w * 32 + (lane & 31);
  const bool ok = key < end && (!mask || mask[key] != 0);

  f32x16_t dk[DP / 32], dv[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) dk[dt] = dv[dt] = zero16();
  if (tile * 128 < end) {
    u32x4_t k[TL::KB], v[TL::KB];
    load_row_frags<T, DP>((const T*)a.k + key * a.ks.t + b * a.ks.b + hk * a.ks.h, a.D, a.whole & kWholeK, ok, lane, k);
    if (DK)
      load_row_frags<T, DP>((const T*)a.v + key * a.vs.t + b * a.vs.b + hk * a.vs.h, a.D, a.whole & kWholeV, ok, lane,
                            v);
    const float c2 = a.scale * kLog2e;
    const int nt = (a.Tq + NR - 1) / NR, n = nt * a.G;
    Loader<T, DP, NR, 4, DMA> lq, lg;
    const T* q0 = (const T*)a.q + b * a.qs.b + (int64_t)hk * a.G * a.qs.h;
    const T* g0 = (const T*)a.dout + b * a.gs.b + (int64_t)hk * a.G * a.gs.h;
    lq.init(q0, a.qs.t, a.D, a.whole & kWholeQ, nullptr, w, lane);
    lg.init(g0, a.gs.t, a.D, a.whole & kWholeG, nullptr, w, lane);
    float st_l = INFINITY, st_d = 0.f;
    auto fetch = [&](int i, int buf) {
      const int hd = i / nt, t0 = (i - hd * nt) * NR;
      lq.p = q0 + hd * a.qs.h;
      lg.p = g0 + hd * a.gs.h;
      lq.load(t0, a.Tq, lds + buf * 2 * TB);
      lg.load(t0, a.Tq, lds + buf * 2 * TB + TB);
      if (threadIdx.x < NR) {
        const int t = t0 + threadIdx.x;
        st_l = INFINITY;
        st_d = 0.f;
        if (t < a.Tq) {
          const int64_t li = ((int64_t)b * a.Hq + hk * a.G + hd) * a.Tq + t;
          const float x = a.lse[li];
          if (x != -INFINITY) st_l = x * kLog2e - kInExponent<T>;
          st_d = a.delta[li];
        }
      }
    };
    auto keep = [&](int buf) {
      if (threadIdx.x < NR) {
        stat[buf][0][threadIdx.x] = st_l;
        stat[buf][1][threadIdx.x] = st_d;
      }
    };
    fetch(0, 0);
    keep(0);
    for (int i = 0; i < n; ++i) {
      wait_vmem();
      __syncthreads();
      const int buf = i & 1;
      const char* qt = lds + buf * 2 * TB;
      const char* gt = qt + TB;
      if (i + 1 < n) fetch(i + 1, buf ^ 1);
      f32x16_t s = zero16(), dp = zero16();
#pragma unroll
      for (int kb = 0; kb < TL::KB; ++kb) s = Mm<T>::mac(TL::row_frag(qt, 0, kb, lane), k[kb], s);
      if (DK) {
#pragma unroll
        for (int kb = 0; kb < TL::KB; ++kb) dp = Mm<T>::mac(TL::row_frag(gt, 0, kb, lane), v[kb], dp);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4_t L = *(const f32x4_t*)&stat[buf][0][reg_row(4 * j, lane)];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * j + e] = exp_carried<T>(__builtin_fmaf(s[4 * j + e], c2, -L[e]));
      }
      if (DV) {
#pragma unroll
        for (int pb = 0; pb < TL::PB; ++pb) {
          const u32x4_t p = TL::reg_frag(s, pb);
#pragma unroll
          for (int dt = 0; dt < DP / 32; ++dt) dv[dt] = Mm<T>::mac(TL::col_frag(gt, TL::KR * pb, dt, lane), p, dv[dt]);
        }
      }
      if (DK) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4_t d = *(const f32x4_t*)&stat[buf][1][reg_row(4 * j, lane)];
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
      if (i + 1 < n) keep(buf ^ 1);
    }
  }
  if (key >= a.Tk) return;
  if (!ok) {  // keys of no query: zeros, whatever the products of their zeroed rows were
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt) dk[dt] = dv[dt] = zero16();
  }
  if (DK) store_col<T, DP>((T*)a.dk + key * a.dks.t + b * a.dks.b + hk * a.dks.h, dk, a.scale / kCarry<T>,
                   a.D, a.whole & kWholeDk, lane);
  if (DV) store_col<T, DP>((T*)a.dv + key * a.dvs.t + b * a.dvs.b + hk * a.dvs.h, dv, 1.f / kCarry<T>, a.D, a.whole & kWholeDv, lane);
}

// ---------------------------------------------------------------------------
template <typename T, int DP, bool DMA>
static hipError_t attend_bwd_t(const AttendPlan& p, const AttendArgs& a0, hipStream_t s) {
  AttendArgs a = a0;
  constexpr int C = Tile<T, DP>::C;
  if (a.M > 0) {
    const size_t lds = (size_t)4 * dq_keys<T, DP>() * C * 16;
    a.tiles = (int)((a.M + 127) / 128);
    const unsigned grid = attend_grid(&a);
    const hipError_t e = allow_lds((const void*)attend_dq_kernel<T, DP, DMA>, lds);
    if (e != hipSuccess) return e;
    attend_dq_kernel<T, DP, DMA><<<grid, 256, lds, s>>>(a);
  }
  if (a.Tk > 0) {
    const size_t lds = (size_t)4 * 32 * C * 16;
    a.tiles = (a.Tk + 127) / 128;
    const unsigned grid = attend_grid(&a);
    if constexpr (DP * sizeof(T) > 512) {
      hipError_t e = allow_lds((const void*)attend_dkv_kernel<T, DP, DMA, true, false>, lds);
      if (e == hipSuccess) e = allow_lds((const void*)attend_dkv_kernel<T, DP, DMA, false, true>, lds);
      if (e != hipSuccess) return e;
      attend_dkv_kernel<T, DP, DMA, true, false><<<grid, 256, lds, s>>>(a);
      attend_dkv_kernel<T, DP, DMA, false, true><<<grid, 256, lds, s>>>(a);
    } else {
      const hipError_t e = allow_lds((const void*)attend_dkv_kernel<T, DP, DMA, true, true>, lds);
      if (e != hipSuccess) return e;
      attend_dkv_kernel<T, DP, DMA, true, true><<<grid, 256, lds, s>>>(a);
    }
  }
  return hipGetLastError();
}

hipError_t launch_attend_bwd(const AttendPlan& p, const AttendArgs& a, hipStream_t s) {
  if (a.B == 0) return hipSuccess;
  Timed tm(8, s);
#define ATTEND_DP(T, N) \
  if (p.DP == N) return p.dma ? attend_bwd_t<T, N, true>(p, a, s) : attend_bwd_t<T, N, false>(p, a, s)
#define ATTEND_T(T) \
  ATTEND_DP(T, 32); ATTEND_DP(T, 64); ATTEND_DP(T, 96); ATTEND_DP(T, 128); ATTEND_DP(T, 192); ATTEND_DP(T, 256)
  if (p.dtype == LSTM_F32) { ATTEND_T(float); }
  if (p.dtype == LSTM_BF16) { ATTEND_T(bf16_t); }
  if (p.dtype == LSTM_F16) { ATTEND_T(f16_t); }
  return hipErrorInvalidValue;
}

}  // namespace lstm
