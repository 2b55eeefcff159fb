// linattn_common.hpp -- linear attention with a decay for each head, by chunks
// of 32 steps (gfx950).
//
//   S_t = a S_{t-1} + k_t v_t^T,  o_t = scale q_t S_t
//
// Over a chunk of n steps that starts from S,
//   o_i = scale ( a^(i+1) q_i S + sum_{j<=i} a^(i-j) (q_i . k_j) v_j )
//   S'  = a^n S + sum_j a^(n-1-j) k_j v_j^T.
// The gradients are the same recurrence with the parts exchanged.  With
// R_t = a R_{t+1} + scale q_t do_t^T, the gradient of S_t,
//   dq_t = scale S_t do_t     (rows do, keys v, values k, state S^T)
//   dk_t = R_t v_t            (backwards in time: rows v, keys do, values q, state R^T)
//   dv_t = R_t^T k_t          (backwards in time: rows k, keys q, values do, state R)
// so that one kernel is all four: a "run" has rows a, keys k and values v,
// out_i = scale (inner_i + state part), and a direction of time.  Backwards,
// the state X that is carried to a chunk has been through its step's decay
// already (what R_T = dstate stands for):
//   out_i = scale ( a^(n-1-i) a_i X + sum_{j>=i} a^(j-i) (a_i . k_j) v_j )
//   X'    = a^n X + sum_j a^(j+1) k_j v_j^T,
// with X in units of 1 / scale.
#pragma once
#include "attend_common.hpp"
#include "model_internal.hpp"

namespace lstm {

// A work-group walks over the chunks of a (sequence, head of a, block of 32 NW
// columns of v); each of its NW waves owns 32 of the columns and the state's
// DK x 32 part of them, in the accumulators of the matrix cores:
//   P^T = K A^T            rows j down the registers, column i = lane: weighted
//                          and rounded they are an operand as they stand
//   O^T = S^T A^T + V^T P^T
//   S  += K^T (V weighted)
// Every wave computes P for itself: 8 of its 34 products (rows of 128 16-bit
// values), which costs less than passing it round with two more barriers.
// The state as the operand of the first product of O^T has its k index down
// the registers too; in 16 bits the columns of K are read in the order (bits 2
// and 3 of the index exchanged) that leaves its rows in row_frag's order.
template <typename T, int DP>
struct StateTile : Tile<T, DP> {
  using TL = Tile<T, DP>;
  // col_frag whose lanes hold the columns in the state's order
  __device__ __forceinline__ static u32x4_t col_frag_state(const char* lds, int row0, int dt, int lane) {
    if constexpr (sizeof(T) == 2) {
      u32x4_t out;
      const int L = lane & 15, r = 4 * (lane >> 5) + (L >> 2), c = ((L & 1) << 1) | ((L >> 1) & 1);
      const int d = 32 * dt + 16 * ((lane >> 4) & 1) + 4 * c;
      const char* p = lds + row0 * TL::C * 16 + TL::chunk_at(r, d >> 3) + (d & 7) * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const s16x4_lds_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_t*)(p + h * 8 * TL::C * 16));
        const uint2 u = __builtin_bit_cast(uint2, v);
        out[2 * h] = u.x;
        out[2 * h + 1] = u.y;
      }
      return out;
    } else {
      return TL::col_frag(lds, row0, dt, lane);
    }
  }
  // row of the state in register i of a tile
  __device__ __forceinline__ static int state_row(int i, int lane) {
    if constexpr (sizeof(T) == 2) return 16 * (i >> 3) + 8 * (lane >> 5) + (i & 7);
    else return reg_row(i, lane);
  }
};

// Row of the k-index element e (register order) of k-block pb across the rows.
template <typename T>
__device__ __forceinline__ int frag_row(int pb, int e, int lane) {
  if constexpr (sizeof(T) == 2) return 16 * pb + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
  else return 8 * pb + 4 * (lane >> 5) + e;
}

// decay^e of a whole e >= 0; ld2 = log2 of the decay, -inf for 0.
__device__ __forceinline__ float power(float ld2, int e) { return e == 0 ? 1.f : __builtin_amdgcn_exp2f(ld2 * (float)e); }
__device__ __forceinline__ float log2_decay(const float* log_decay, int h) {
  const float x = log_decay[h];
  return (x > 0.f ? 0.f : x) * kLog2e;
}

// The power of two that brings the largest of a wave's values to [2^13, 2^14)
// (1 where there is none, or it is not finite): operands in fp16 are scaled by
// it, so that sums beyond 65504 and values among its denormals keep their bits.
__device__ __forceinline__ float lift_of(float most) {
  auto from = [&](auto ctl) {
    const uint32_t v = __float_as_uint(most);
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, decltype(ctl)::value, 0xf, 0xf, false));
  };
  using std::integral_constant;
  most = fmaxf(most, from(integral_constant<int, 0xB1>{}));   // quad_perm 1,0,3,2
  most = fmaxf(most, from(integral_constant<int, 0x4E>{}));   // quad_perm 2,3,0,1
  most = fmaxf(most, from(integral_constant<int, 0x124>{}));  // row_ror:4
  most = fmaxf(most, from(integral_constant<int, 0x128>{}));  // row_ror:8
  const auto r16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(most), __float_as_uint(most), false, false);
  most = fmaxf(__uint_as_float(r16[0]), __uint_as_float(r16[1]));
  most = fmaxf(most, other_half(most));
  const uint32_t e = __float_as_uint(most) >> 23;  // exponent (most >= 0)
  const uint32_t r = e == 0 || e == 255 ? 127u : 127u + 13u + 127u - e;
  return __uint_as_float(__builtin_amdgcn_readfirstlane((r < 1 ? 1u : r > 253 ? 253u : r) << 23));
}

template <int N>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Loads a tensor's rows 0 .. `rows` - 1 (row r at p + r st) into rows `shift` ..
// of a tile of 32 at an LDS address with NW waves; the tile's other rows and
// values past D become zeros.  DMA:
// straight into LDS (rows of whole 16-byte chunks, st >= D, 32 st below 2^31
// bytes); else chunk by chunk through registers.
template <typename T, int DP, int NW, bool DMA>
struct Rows32 {
  using TL = Tile<T, DP>;
  static constexpr int kLoads = 32 * TL::C / 64 / NW;  // loads of 1 KB a wave
  static_assert(32 * TL::C / 64 % NW == 0, "every wave has as many");
  int64_t st;
  int D, whole, w, lane;
  uint32_t off[kLoads];  // DMA: byte offset of this lane's chunk of each load
  __device__ __forceinline__ void init(int64_t st_, int D_, int whole_, int w_, int lane_) {
    st = st_; D = D_; whole = whole_; w = w_; lane = lane_;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = (j * NW + w) * 64 + lane, r = i / TL::C, c = (i % TL::C) ^ TL::swizzle(r);
      off[j] = c * 16 < D * (int)sizeof(T) ? (uint32_t)(r * (int)st * (int)sizeof(T) + c * 16) : kNoRow;
    }
  }
  __device__ __forceinline__ void load(const T* p, int rows, int shift, uint32_t lds) const {
    if constexpr (DMA) {
      const int bytes = rows > 0 ? (int)(((rows - 1) * (int)st + D) * (int)sizeof(T)) : 0;
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00020000);
#pragma unroll
      // (a row before the first: an offset below 0, past the descriptor's end)
      for (int j = 0; j < kLoads; ++j)
        lds_dma16_at<false>(r, lds + (j * NW + w) * 1024, off[j] - (uint32_t)(shift * (int)st * (int)sizeof(T)), 0);
    } else {
      typedef __attribute__((address_space(3))) u32x4_t lds_vec_t;
      for (int j = 0; j < kLoads; ++j) {
        const int i = (j * NW + w) * 64 + lane, r = i / TL::C, c = (i % TL::C) ^ TL::swizzle(r);
        u32x4_t v = {0, 0, 0, 0};
        if (r >= shift && r - shift < rows) v = load_chunk<T>(p + (r - shift) * st, c * vec_of<T>(), D, whole != 0);
        *(lds_vec_t*)(uintptr_t)(lds + i * 16) = v;
      }
    }
  }
};

constexpr int kAheadRows = 6, kAheadCols = 4;  // fragments read ahead of their products
// What a launch does: the run (kOne: one head of keys a state, kSum: several),
// or the segments' own sums alone, without rows a and outputs.
enum { kOne = 0, kSum = 1, kState = 2 };
template <typename T, int DP, int NW, int KIND> constexpr int lin_stage_bytes() {
  return (KIND == kState ? 1 : 2) * Tile<T, DP>::kBytes32 + Tile<T, 32 * NW>::kBytes32;
}
// Stages of LDS: three where two work-groups of them fit a compute unit or
// nothing is gained by fewer.
template <typename T, int DP, int NW, int KIND> constexpr int lin_stages() {
  return 3 * lin_stage_bytes<T, DP, NW, KIND>() <= 150 * 1024 ? 3 : 2;
}

template <typename T, int DP, int NW, bool DMA, int KIND>
__global__ void __launch_bounds__(64 * NW, DP * sizeof(T) > 256 ? 1 : 2) linattn_kernel(LinArgs args) {
  using TK = StateTile<T, DP>;
  using TV = Tile<T, 32 * NW>;
  constexpr bool kHalf = std::is_same<T, f16_t>::value;
  constexpr int NST = lin_stages<T, DP, NW, KIND>(), kStage = lin_stage_bytes<T, DP, NW, KIND>();
  constexpr bool state_only = KIND == kState;
  constexpr int kAtK = state_only ? 0 : TK::kBytes32, kAtV = kAtK + TK::kBytes32;  // of a stage
  constexpr int NDT = DP / 32, PB = TK::PB, EB = vec_of<T>();
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // which run, and which (sequence, head, columns, segment) of it
  int64_t u = blockIdx.x;
  int which = 0;
  while (which + 1 < args.runs && u >= args.run[which + 1].group0) ++which;
  const LinRun& x = args.run[which];
  u -= x.group0;
  const int heads = state_only ? args.Hs : x.Ha;
  const int dvb = (int)(u % x.dv_blocks);
  u /= x.dv_blocks;
  const int h = (int)(u % heads);
  u /= heads;
  const int order = (int)(u % args.segs_of_launch);  // in the order of the run's time
  const int b = (int)(u / args.segs_of_launch);
  const int hs = state_only ? h : h / x.ga;
  const int seg = x.rev ? args.segs - 1 - order : order;
  int64_t end = args.T;
  if (args.len) {
    const int64_t l = args.len[b];
    end = l < 0 ? 0 : l < args.T ? l : args.T;
  }
  const int64_t r0 = (int64_t)seg * args.seg_rows;
  int64_t r1 = r0 + args.seg_rows < end ? r0 + args.seg_rows : end;
  if (r1 < r0) r1 = r0;
  const int n_chunks = (int)((r1 - r0 + 31) >> 5);
  const int rev = x.rev, gb = KIND == kOne ? 1 : x.gb;
  const float ld2 = log2_decay(args.log_decay, hs);
  const int dv0 = dvb * 32 * NW, cols = x.DV - dv0;  // (cols > 0)

  Rows32<T, DP, NW, DMA> la, lk;
  Rows32<T, 32 * NW, NW, DMA> lv;
  la.init(x.as.t, x.DK, x.whole & kWholeQ, w, lane);
  lk.init(x.ks.t, x.DK, x.whole & kWholeK, w, lane);
  lv.init(x.vs.t, cols < 32 * NW ? cols : 32 * NW, x.whole & kWholeV, w, lane);
  const T* a0 = (const T*)x.a + b * x.as.b + h * x.as.h;
  const T* k0 = (const T*)x.k + b * x.ks.b + (int64_t)hs * gb * x.ks.h;
  const T* v0 = (const T*)x.v + b * x.vs.b + (int64_t)hs * gb * x.vs.h + dv0;
  constexpr int kLoads = (state_only ? 0 : decltype(la)::kLoads) + decltype(lk)::kLoads + decltype(lv)::kLoads;

  // the state this wave carries: tile dt, register i
  const int64_t head = (int64_t)b * args.Hs + hs, state_size = (int64_t)x.DK * x.DV;
  f32x16_t S[NDT];
  {
    const float* in = x.s_in ? x.s_in + head * state_size : nullptr;
    int s_dk = (int)x.s_dk, s_dv = (int)x.s_dv;
    float by = x.in_by;
    if (args.segs > 1) {
      in = state_only ? nullptr : x.seg + (head * args.segs + order) * state_size;
      s_dk = x.DV; s_dv = 1;
      by = 1.f;
    }
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)in, 0, in ? (int)state_size * 4 : 0, 0x00020000);
    const int dv = dv0 + 32 * w + (lane & 31);
#pragma unroll
    for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = 32 * dt + TK::state_row(i, lane);
        const uint32_t at = d < x.DK && dv < x.DV ? (uint32_t)(d * s_dk + dv * s_dv) * 4 : kNoRow;
        S[dt][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0)) * by;
      }
  }
  float lift = 1.f;  // fp16: S holds the state times this power of two

  // Weights of P (row j = reg_row, column i = lane) and of V in the state's sum.
  // They count from the chunk's end forwards in time and from its beginning
  // backwards, so a chunk of fewer than 32 steps lies at that end of its tiles.
  const int ri = lane & 31;
  float wp[16], wv[PB][EB];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int j = reg_row(i, lane), e = rev ? j - ri : ri - j;
    wp[i] = e < 0 ? 0.f : power(ld2, e);
  }
#pragma unroll
  for (int pb = 0; pb < PB; ++pb)
#pragma unroll
    for (int e = 0; e < EB; ++e) {
      const int j = frag_row<T>(pb, e, lane);
      wv[pb][e] = power(ld2, rev ? j + 1 : 31 - j);
    }
  // the state of this work-group reaches an output in fp32
  const bool state_out = x.s_out != nullptr && (state_only || h % x.ga == 0);
  f32x16_t O = zero16();
  const int iters = n_chunks * gb;
  // iteration it: chunk it / gb (in the order of time), head it % gb of the keys
  int lc = 0, lg = 0;  // of the next load
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void_t*)lds;
  auto load = [&](int slot) __attribute__((always_inline)) {
    const uint32_t at = lds0 + slot * kStage;
    const int64_t row0 = r0 + 32 * (int64_t)(rev ? n_chunks - 1 - lc : lc);
    const int rows = (int)(r1 - row0 < 32 ? r1 - row0 : 32);
    const int shift = rev ? 0 : 32 - rows;
    if constexpr (!state_only) la.load(a0 + row0 * x.as.t, rows, shift, at);
    lk.load(k0 + lg * x.ks.h + row0 * x.ks.t, rows, shift, at + kAtK);
    lv.load(v0 + lg * x.vs.h + row0 * x.vs.t, rows, shift, at + kAtV);
    if (++lg == gb) {
      lg = 0;
      ++lc;
    }
  };
#pragma unroll
  for (int i = 0; i < NST - 1; ++i)
    if (i < iters) load(i);

  T* out = (T*)x.out + b * x.os.b + h * x.os.h + dv0 + 32 * w;
  const int out_cols = cols - 32 * w;  // (may be below 0: no columns)
  const float scale = args.scale;
  // O of the chunk whose rows begin at row0, times scale
  auto store = [&](int64_t row0) __attribute__((always_inline)) {
    const int shift = rev || r1 - row0 >= 32 ? 0 : 32 - (int)(r1 - row0);
    const int64_t row = row0 + ri - shift;
    const bool there = ri >= shift && row < r1;
    T* p = out + row * x.os.t;
    if ((x.whole & kWholeO) && out_cols >= 32) {
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t lo[2], hi[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            lo[c] = pack2<T>(O[8 * i + 2 * c] * scale, O[8 * i + 2 * c + 1] * scale);
            hi[c] = pack2<T>(O[8 * i + 4 + 2 * c] * scale, O[8 * i + 4 + 2 * c + 1] * scale);
          }
          const auto s0 = __builtin_amdgcn_permlane32_swap(lo[0], hi[0], false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(lo[1], hi[1], false, false);
          const u32x4_t q = {s0[0], s1[0], s0[1], s1[1]};
          if (there) *(u32x4_t*)(p + 16 * i + 8 * (lane >> 5)) = q;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (there)
            *(f32x4_t*)(p + reg_row(4 * i, lane)) = f32x4_t{O[4 * i] * scale, O[4 * i + 1] * scale, O[4 * i + 2] * scale, O[4 * i + 3] * scale};
      }
    } else if (there) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = reg_row(i, lane);
        if (d < out_cols) p[d] = Elem<T>::from_f(as_f32(O[i] * scale));
      }
    }
  };

  int c = 0, g = 0;
  for (int it = 0; it < iters; ++it) {
    // this iteration's rows have come; those of the next (NST = 3) may be on their way
    if (NST == 2 || it + 1 == iters) stage_barrier<0>();
    else stage_barrier<kLoads>();
    if (!state_only && it > 0 && g == 0) {  // the chunk before
      const int64_t row0 = r0 + 32 * (int64_t)(rev ? n_chunks - c : c - 1);
      store(row0);
    }
    if (it + NST - 1 < iters) load((it + NST - 1) % NST);
    const int ln = tile_lane<true>(lane);  // (fragment addresses kept over the iterations would take the registers)
    const char* at = lds + (it % NST) * kStage;
    const char *ta = at, *tk = at + kAtK, *tv = at + kAtV;
    const int64_t row0 = r0 + 32 * (int64_t)(rev ? n_chunks - 1 - c : c);
    const int n = (int)(r1 - row0 < 32 ? r1 - row0 : 32);

    if constexpr (!state_only) {
      f32x16_t P = zero16();
      float undo = 1.f;
      // rows of a and k in turn, k-block by k-block
      u32x4_t af;
      Ahead<2 * TK::KB, kAheadRows> rows;
      auto read_rows = [&](int f) __attribute__((always_inline)) { return TK::row_frag(f & 1 ? tk : ta, 0, f >> 1, ln); };
      if (KIND == kOne || g == 0) {
        float by = 1.f;
        if constexpr (kHalf) {
          float most = 0.f;
#pragma unroll
          for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(S[dt][i]));
          by = lift_of(most);
          undo = 1.f / (by * lift);
        }
        O = zero16();
        constexpr int kPer = sizeof(T) == 2 ? 2 : 4;  // k-blocks of a tile of the state
        rows.start(read_rows);
        rows.run(read_rows, [&](int f, u32x4_t q) __attribute__((always_inline)) {
          const int kb = f >> 1;
          if (!(f & 1)) {
            af = q;
            return;
          }
          u32x4_t sf;
          if constexpr (kHalf) {
            f32x16_t s;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[8 * (kb % kPer) + i] = S[kb / kPer][8 * (kb % kPer) + i] * by;
            sf = TK::reg_frag(s, kb % kPer);
          } else {
            sf = TK::reg_frag(S[kb / kPer], kb % kPer);
          }
          P = Mm<T>::mac(q, af, P);
          O = Mm<T>::mac(sf, af, O);
        });
        const int e = rev ? n - 1 - ri : ri + 1 - (32 - n);
        const float f = power(ld2, e < 0 ? 0 : e) * undo;
#pragma unroll
        for (int i = 0; i < 16; ++i) O[i] *= f;
      } else {
        rows.start(read_rows);
        rows.run(read_rows, [&](int f, u32x4_t q) __attribute__((always_inline)) {
          if (f & 1) P = Mm<T>::mac(q, af, P);
          else af = q;
        });
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) P[i] *= wp[i];
      float by = 1.f;
      if constexpr (kHalf) {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(P[i]));
        by = lift_of(most);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          P[i] *= by;
          O[i] *= by;
        }
      }
#pragma unroll
      for (int pb = 0; pb < PB; ++pb) O = Mm<T>::mac(TV::col_frag(tv, TK::KR * pb, w, ln), TK::reg_frag(P, pb), O);
      if constexpr (kHalf) {
        const float un = 1.f / by;
#pragma unroll
        for (int i = 0; i < 16; ++i) O[i] *= un;
      }
    }

    // the state's sum: V weighted, in 16 bits as two numbers (fp16 to 2^-22,
    // bf16 to 2^-17) and in bf16 as a third where the state is an fp32 output
    float f[PB][EB];
#pragma unroll
    for (int pb = 0; pb < PB; ++pb) {
      unpack<T>(TV::col_frag(tv, TK::KR * pb, w, ln), f[pb]);
#pragma unroll
      for (int e = 0; e < EB; ++e) f[pb][e] *= wv[pb][e];
    }
    float keep = KIND == kOne || g == 0 ? power(ld2, n) : 1.f;
    if constexpr (kHalf) {
      float most = 0.f;
#pragma unroll
      for (int pb = 0; pb < PB; ++pb)
#pragma unroll
        for (int e = 0; e < EB; ++e) most = fmaxf(most, fabsf(f[pb][e]));
      const float to = lift_of(most);
      keep *= to / lift;
      lift = to;
#pragma unroll
      for (int pb = 0; pb < PB; ++pb)
#pragma unroll
        for (int e = 0; e < EB; ++e) f[pb][e] *= to;
    }
#pragma unroll
    for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) S[dt][i] *= keep;
    constexpr int kParts = sizeof(T) == 4 ? 1 : kHalf ? 2 : 3;
    u32x4_t vw[PB][kParts];
#pragma unroll
    for (int pb = 0; pb < PB; ++pb) {
      vw[pb][0] = pack<T>(f[pb]);
#pragma unroll
      for (int i = 1; i < kParts; ++i) {  // what the number before has rounded away
        float r[EB];
        unpack<T>(vw[pb][i - 1], r);
#pragma unroll
        for (int e = 0; e < EB; ++e) f[pb][e] -= r[e];
        vw[pb][i] = pack<T>(f[pb]);
      }
    }
    Ahead<PB * NDT, kAheadCols> kcols;
    auto read_cols = [&](int i) __attribute__((always_inline)) { return TK::col_frag_state(tk, TK::KR * (i / NDT), i % NDT, ln); };
    kcols.start(read_cols);
    kcols.run(read_cols, [&](int i, u32x4_t kf) __attribute__((always_inline)) {
      f32x16_t& s = S[i % NDT];
      s = Mm<T>::mac(kf, vw[i / NDT][0], s);
      if constexpr (kParts > 1) s = Mm<T>::mac(kf, vw[i / NDT][1], s);
      if constexpr (kParts > 2)
        if (state_out) s = Mm<T>::mac(kf, vw[i / NDT][2], s);
    });
    if (++g == gb) {
      g = 0;
      ++c;
    }
  }
  if (!state_only) {
    if (iters > 0) store(r0 + 32 * (int64_t)(rev ? 0 : n_chunks - 1));
    // steps past the end
    const int64_t top = r0 + args.seg_rows < args.T ? r0 + args.seg_rows : args.T;
    for (int64_t row = (r1 > r0 ? r1 : r0) + w; row < top; row += NW) {
      T* p = (T*)x.out + b * x.os.b + h * x.os.h + dv0 + row * x.os.t;
      for (int d = lane; d < 32 * NW && d < cols; d += 64) p[d] = Elem<T>::from_f(0.f);
    }
  }
  // the state after the run, or the segment's own sum
  float* to = nullptr;
  int s_dk = (int)x.s_dk, s_dv = (int)x.s_dv;
  float by = x.out_by;
  if (state_only) {
    to = x.seg + (head * args.segs + order) * state_size;
    s_dk = x.DV; s_dv = 1;
    by = 1.f;
  } else if (state_out && order == args.segs - 1) {
    to = x.s_out + head * state_size;
  }
  if (to) {
    if constexpr (kHalf) by /= lift;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)to, 0, (int)state_size * 4, 0x00020000);
    const int ln = tile_lane<true>(lane), dv = dv0 + 32 * w + (ln & 31);
#pragma unroll
    for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = 32 * dt + TK::state_row(i, ln);
        const uint32_t at = d < x.DK && dv < x.DV ? (uint32_t)(d * s_dk + dv * s_dv) * 4 : kNoRow;
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[dt][i] * by), r, at, 0, 0);
      }
  }
}

template <typename T, int DP, int NW, bool DMA, int KIND>
static hipError_t linattn_launch(const LinArgs& a, unsigned groups, hipStream_t s) {
  const size_t bytes = (size_t)lin_stages<T, DP, NW, KIND>() * lin_stage_bytes<T, DP, NW, KIND>();
  const hipError_t e = allow_lds<linattn_kernel<T, DP, NW, DMA, KIND>>(bytes);
  if (e != hipSuccess) return e;
  Timed timed(10, s);
  linattn_kernel<T, DP, NW, DMA, KIND><<<dim3(groups), 64 * NW, bytes, s>>>(a);
  return hipGetLastError();
}
template <typename T, int DP, int NW, bool DMA>
static hipError_t linattn_kind(const LinArgs& a, unsigned groups, hipStream_t s) {
  if (a.state_only) return linattn_launch<T, DP, NW, DMA, kState>(a, groups, s);
  int gb = 1;
  for (int i = 0; i < a.runs; ++i) gb = a.run[i].gb > gb ? a.run[i].gb : gb;
  return gb > 1 ? linattn_launch<T, DP, NW, DMA, kSum>(a, groups, s) : linattn_launch<T, DP, NW, DMA, kOne>(a, groups, s);
}
template <typename T, int DP, int NW>
static hipError_t linattn_loads(const LinArgs& a, int dma, unsigned groups, hipStream_t s) {
  return dma ? linattn_kind<T, DP, NW, true>(a, groups, s) : linattn_kind<T, DP, NW, false>(a, groups, s);
}
template <typename T>
static hipError_t linattn_of(const LinArgs& a, int dp, int nw, int dma, unsigned groups, hipStream_t s) {
  switch (dp + nw) {
    case 64 + 2: return linattn_loads<T, 64, 2>(a, dma, groups, s);
    case 64 + 4: return linattn_loads<T, 64, 4>(a, dma, groups, s);
    case 128 + 2: return linattn_loads<T, 128, 2>(a, dma, groups, s);
    case 128 + 4: return linattn_loads<T, 128, 4>(a, dma, groups, s);
    case 256 + 2: return linattn_loads<T, 256, 2>(a, dma, groups, s);
    default: return linattn_loads<T, 256, 4>(a, dma, groups, s);
  }
}

}  // namespace lstm
