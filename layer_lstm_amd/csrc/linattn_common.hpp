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
// and a direction of time.  Backwards, the state X that is carried to a chunk has
// been through its step's decay already (what dstate stands for), and has the
// scale in it:
//   out_i = a^(n-1-i) a_i X + scale sum_{j>=i} a^(j-i) (a_i . k_j) v_j
//   X'    = a^n X + scale sum_j a^(j+1) k_j v_j^T.
#pragma once
#include "attend_common.hpp"
#include "linattn_decay.hpp"
#include "model_internal.hpp"

namespace lstm {

// A work-group walks over the chunks of a (sequence, head of a, block of 32 NW
// columns of v).  Its NW KS waves own 32 of the columns and a KS-th of the rows
// of the state each, DK / KS x 32 in the accumulators of the matrix cores:
//   P^T = K A^T            rows j down the registers, column i = lane: weighted
//                          and rounded they are an operand as they stand
//   O^T = S^T A^T + V^T P^T
//   S  += K^T (V weighted)
// Every wave computes P for itself (over its own d: the waves of the same
// columns have parts of O, which they add up through LDS; the next chunk's
// barrier is theirs too).  Passing P round instead would cost two barriers for
// 8 of a wave's 34 products (rows of 128 16-bit values, KS = 1).
//
// What bounds it: instruction issue.  A chunk of 32 steps of 128-value bf16 rows
// is some 300 vector instructions a wave and column tile (weighing and splitting
// V 80 to 120, scaling and rounding the state 96, P and O 60) beside its 34
// matrix instructions, which keep the matrix units 24 to 34 % busy, and the
// memory's traffic is below half the copy's rate forwards (8 sequences, 16 heads
// of 128, 4096 steps: 185 us, 2.9 TB/s; the same with rows that stay in L2) and
// 4.2 TB/s backwards (355 us).  fp32 is bound by the chain of its matrix
// instructions.
// The state as the operand of the first product of O^T has its k index down
// the registers too; in 16 bits the columns of K are read in the order (bits 2
// and 3 of the index exchanged) that leaves its rows in row_frag's order.
// In 16 bits P and the state are operands rounded once to the storage type, as
// the rows are that they multiply (both are summed and carried in fp32).  The
// outputs' errors are 2.35e-3 of the norm in bf16 so, where the output's own
// rounding is 1.66e-3; with P as two numbers 2.2 to 2.3e-3, the state 1.73 to
// 1.84e-3, both 1.66e-3, at 3, 10 and 16 % of the forward's time and 3, 18 and
// 22 % of the backward's (8 sequences, 16 heads of 128, 4096 steps).  They stay
// at one.
//
// Fragment addresses.  Rows are multiples of 128 bytes and tiles of 1 KB, so a
// fragment's chunk is a lane's first one with bits flipped (the swizzle is an
// exclusive or) and constants added: three registers hold a lane's part of all.
typedef __attribute__((address_space(3))) u32x4_t lds_vec_t;
typedef __attribute__((address_space(3))) uint32_t lds_word_t;

template <typename T, int DP>
struct StateTile : Tile<T, DP> {
  using TL = Tile<T, DP>;
  static_assert(TL::C % 8 == 0, "rows of whole 128 bytes");
  static constexpr int kRow = TL::C * 16;
  // Tile::row_frag(row0 = 0, kb): this lane's first chunk, and a fragment from
  // the tile's address plus it
  __device__ __forceinline__ static uint32_t row_first(int lane) {
    return (lane & 31) * kRow + (((lane >> 5) ^ TL::swizzle(lane & 31)) * 16);
  }
  __device__ __forceinline__ static u32x4_t row_at(uint32_t at, int kb) {
    return *(lds_vec_t*)(uintptr_t)((at ^ (32 * (kb & 3))) + 128 * (kb >> 2));
  }
  // Tile::col_frag: the same; in 16 bits with `state`, the columns in the
  // state's order
  __device__ __forceinline__ static uint32_t col_first(int lane, bool state) {
    if constexpr (sizeof(T) == 2) {
      const int L = lane & 15, r = 4 * (lane >> 5) + (L >> 2), c = state ? ((L & 1) << 1) | ((L >> 1) & 1) : L & 3;
      return r * kRow + (((2 * ((lane >> 4) & 1) + (c >> 1)) ^ TL::swizzle(r)) * 16) + (c & 1) * 8;
    } else {
      const int r = 4 * (lane >> 5);
      return r * kRow + ((((lane & 31) >> 2) ^ TL::swizzle(r)) * 16) + (lane & 3) * 4;
    }
  }
  __device__ __forceinline__ static u32x4_t col_at(uint32_t at, int row0, int dt) {
    u32x4_t out;
    if constexpr (sizeof(T) == 2) {
      const uint32_t p = (at ^ (64 * (dt & 1))) + 128 * (dt >> 1) + row0 * kRow;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 u = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_t*)(uintptr_t)(p + h * 8 * kRow)));
        out[2 * h] = u.x;
        out[2 * h + 1] = u.y;
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s)  // swizzle(r + s) = swizzle(r) with these bits flipped, r a multiple of 4
        out[s] = *(lds_word_t*)(uintptr_t)((at ^ ((s & 1) * 64 | (s >> 1) * 16)) + (row0 + s) * kRow + 128 * dt);
    }
    return out;
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

// fp16: operands are scaled by powers of two, so that sums beyond 65504 and
// values among its denormals keep their bits.  Columns of V, and with them of the
// state, and rows of P each have their own (a lane holds one), so that none loses
// its bits to a larger one beside it; the state as an operand has one for all of
// a wave's (a column counts from 2^-27 of the largest on, and its outputs are
// fp16).
// The power of two that brings x (>= 0) to [2^13, 2^14); 1 where x is 0 or not
// finite; from 2^lo to 2^hi.
__device__ __forceinline__ uint32_t lift_bits(float x, int lo, int hi) {
  const int e = (int)(__float_as_uint(x) >> 23), r = e == 0 || e == 255 ? 127 : 127 + 13 + 127 - e;
  return (uint32_t)(r < 127 + lo ? 127 + lo : r > 127 + hi ? 127 + hi : r);
}
__device__ __forceinline__ float power_of_two(uint32_t bits) { return __uint_as_float(bits << 23); }
__device__ __forceinline__ float inverse(float power) { return __uint_as_float((254u << 23) - __float_as_uint(power)); }
// The largest of a wave's values.
__device__ __forceinline__ float wave_max(float most) {
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
  return fmaxf(most, other_half(most));
}

// The product whose zeros make zero of anything, NaN and infinities too
// (v_mul_legacy_f32; the intrinsic has no builtin).
__device__ float mul_zero(float a, float b) __asm("llvm.amdgcn.fmul.legacy");

// sum, or NaN where one of the 16 bytes' values is not finite.
template <typename T>
__device__ __forceinline__ float add_zeros(u32x4_t v, float sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = v[i];  // (a bit cast of v[i] itself takes the vector's first element)
    if constexpr (std::is_same<T, bf16_t>::value) {
      typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
      sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(pair_t, word), __builtin_bit_cast(pair_t, 0u), sum, false);
    } else if constexpr (std::is_same<T, f16_t>::value) {
      typedef _Float16 pair_t __attribute__((ext_vector_type(2)));
      sum = __builtin_amdgcn_fdot2(__builtin_bit_cast(pair_t, word), __builtin_bit_cast(pair_t, 0u), sum, false);
    } else {
      sum = __builtin_fmaf(__uint_as_float(word), 0.f, sum);
    }
  }
  return sum;
}
// Zeros in place of a fragment's values that are not finite; `edge` moves to the
// row of each (frag_row) that is before it, or behind it with `rev`.
template <typename T>
__device__ __forceinline__ u32x4_t finite_only(u32x4_t v, int pb, int lane, bool rev, int* edge) {
  constexpr uint32_t kExponent = sizeof(T) == 4 ? 0x7f800000u : std::is_same<T, f16_t>::value ? 0x7c00u : 0x7f80u;
  constexpr int kEach = 4 / (int)sizeof(T), kBits = 32 / kEach;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      const uint32_t word = v[i];
      if (((word >> (kBits * h)) & kExponent) == kExponent) {
        const int row = frag_row<T>(pb, kEach * i + h, lane);
        *edge = rev ? (row > *edge ? row : *edge) : (row < *edge ? row : *edge);
        v[i] = kEach == 1 ? 0u : word & (h ? 0xffffu : 0xffff0000u);
      }
    }
  return v;
}

template <int N>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Loads a tensor's rows 0 .. `rows` - 1 (row r at p + r st) into rows `shift` ..
// of a tile of 32 at an LDS address with W waves; the tile's other rows and
// values past D become zeros.  DMA: straight into LDS (rows of whole 16-byte
// chunks, st >= D, 64 st below 2^31 bytes); else chunk by chunk through
// registers.
template <typename T, int DP, int W, bool DMA>
struct Rows32 {
  using TL = Tile<T, DP>;
  static constexpr int kAll = 32 * TL::C / 64, kLoads = kAll < W ? 1 : kAll / W;  // loads of 1 KB, of a wave
  // (every wave has as many: where there are fewer than waves, some are made twice)
  static_assert(kAll < W ? W % kAll == 0 : kAll % W == 0, "");
  int64_t st;
  int row_bytes, all_bytes;  // from row to row, of 32 rows
  int D, whole, w, lane;
  uint32_t off[kLoads];  // DMA: byte offset of this lane's chunk of each load
  __device__ __forceinline__ void init(int64_t st_, int D_, int whole_, int w_, int lane_) {
    st = st_; D = D_; whole = whole_; w = w_ % kAll; lane = lane_;
    row_bytes = (int)st * (int)sizeof(T);
    all_bytes = 31 * row_bytes + D * (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = (j * W + w) * 64 + lane, r = i / TL::C, c = (i % TL::C) ^ TL::swizzle(r);
      off[j] = c * 16 < D * (int)sizeof(T) ? (uint32_t)(r * row_bytes + c * 16) : kNoRow;
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void load(const T* p, int rows, int shift, uint32_t lds) const {
    if constexpr (DMA) {
      // (uniform, which the compiler does not see through the loop's selects)
      const uint64_t at = (uint64_t)p;
      const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at), hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
      const int bytes = FULL ? all_bytes : __builtin_amdgcn_readfirstlane(all_bytes - (32 - rows) * row_bytes);
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)hi << 32 | lo), 0, bytes, 0x00020000);
      const uint32_t back = FULL ? 0u : (uint32_t)(shift * row_bytes);  // (a row before the first: an offset below 0, past the end)
#pragma unroll
      for (int j = 0; j < kLoads; ++j) lds_dma16_at<false>(r, lds + (j * W + w) * 1024, off[j] - back, 0);
    } else {
      for (int j = 0; j < kLoads; ++j) {
        const int i = (j * W + w) * 64 + lane, r = i / TL::C, c = (i % TL::C) ^ TL::swizzle(r);
        u32x4_t v = {0, 0, 0, 0};
        if (r >= shift && r - shift < rows) v = load_chunk<T>(p + (r - shift) * st, c * vec_of<T>(), D, whole != 0);
        *(lds_vec_t*)(uintptr_t)(lds + i * 16) = v;
      }
    }
  }
};

constexpr int kAheadRows = 6, kAheadCols = 4;  // fragments read ahead of their products
// What a launch does: runs of one head of a and of k a work-group (kOne), of
// several heads of k and v, whose products add up (kSum), of several heads of a,
// which share a chunk's k, v and the state's update (kMany); or the segments' own sums
// alone, without rows a and outputs (kState).
enum { kOne = 0, kSum = 1, kMany = 2, kState = 3 };
// LDS: stages of an iteration's tiles -- a, k and v; in kMany a alone, and two
// pairs of k and v.  KS > 1: what each wave hands to the other waves of its
// columns, a KS-th of its part of O each, twice.
template <typename T, int DP, int NW, int KS, int KIND>
struct LinLds {
  static constexpr int kA = KIND == kState ? 0 : Tile<T, DP>::kBytes32;
  static constexpr int kKV = Tile<T, DP>::kBytes32 + Tile<T, 32 * NW>::kBytes32;
  static constexpr int kStage = KIND == kMany ? kA : kA + kKV;
  static constexpr int kPass = KS > 1 && KIND != kState ? 2 * NW * KS * (KS - 1) * (4096 / KS) : 0;
  static constexpr int kPairs = KIND == kMany ? 2 * kKV : 0;
  // three stages where they fit a compute unit; two of small tiles, for more
  // work-groups (64 sequences, 16 heads of 64, 256 steps, bf16: forward 27 us,
  // backward 54, with three 28 and 64)
  static constexpr int kStages = (KIND != kMany && kStage <= 12 * 1024) || 3 * kStage + kPairs + kPass > 160 * 1024 ? 2 : 3;
  static constexpr int kAtPairs = kStages * kStage, kAtPass = kAtPairs + kPairs, kBytes = kAtPass + kPass;
  static_assert(kBytes <= 160 * 1024, "a compute unit's LDS");
};

template <typename T, int DP, int NW, int KS, bool DMA, int KIND>
__global__ void __launch_bounds__(64 * NW * KS, DP * sizeof(T) / KS > 256 ? 1 : DP == 64 && KIND == kOne ? 3 : 2)
linattn_kernel(LinArgs args) {
  using TK = StateTile<T, DP>;
  using TV = StateTile<T, 32 * NW>;
  using LL = LinLds<T, DP, NW, KS, KIND>;
  constexpr bool kHalf = std::is_same<T, f16_t>::value, state_only = KIND == kState, kSplit = KS > 1 && !state_only;
  constexpr int NST = LL::kStages;
  constexpr int NDT = DP / 32 / KS, KB = TK::KB / KS, PB = TK::PB, EB = vec_of<T>();
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wave % NW, part = wave / NW;  // columns, rows of the state

  // Which (sequence, head, segment), and which run, columns and head of a of it:
  // the work-groups that read the same rows (columns of a head, heads of a that
  // share a state, the three runs of a backward) are dealt to one XCD, one after
  // the other (work-groups go to the XCDs round robin).
  const uint32_t u = blockIdx.x, slot = (u >> 3) / args.share;
  uint32_t member = (u >> 3) - slot * args.share;
  int which = 0;
  while (which + 1 < args.runs && member >= args.run[which + 1].member0) ++which;
  const LinRun& x = args.run[which];
  member -= x.member0;
  const int dvb = (int)(member % x.dv_blocks), ha = (int)(member / x.dv_blocks);  // (ha: 0 in kMany, kState)
  uint32_t set = slot * 8 + (u & 7);
  if (set >= (uint32_t)args.B * args.Hs * args.segs_of_launch) return;
  const int hs = (int)(set % args.Hs);
  set /= args.Hs;
  const int order = (int)(set % args.segs_of_launch);  // in the order of the run's time
  const int b = (int)(set / args.segs_of_launch);
  const int rev = x.rev, seg = rev ? args.segs - 1 - order : order;
  int64_t end = args.T;
  if (args.len) {
    const int64_t l = args.len[b];
    end = l < 0 ? 0 : l < args.T ? l : args.T;
  }
  const int64_t r0 = (int64_t)seg * args.seg_rows;
  int64_t r1 = r0 + args.seg_rows < end ? r0 + args.seg_rows : end;
  if (r1 < r0) r1 = r0;
  const int steps = (int)(r1 - r0), n_chunks = (steps + 31) >> 5;
  const int heads = KIND == kSum || state_only ? x.gb : KIND == kMany ? x.ga : 1;  // iterations of a chunk
  const Decay decay = Decay::of(args.log_decay, hs);
  const int dv0 = dvb * 32 * NW, cols = x.DV - dv0;  // (cols > 0)

  // the state this wave carries: tile dt, register i
  const int64_t head = (int64_t)b * args.Hs + hs, state_size = (int64_t)x.DK * x.DV;
  f32x16_t S[NDT];
  {
    const float* in = x.s_in ? x.s_in + head * state_size : nullptr;
    int s_dk = (int)x.s_dk, s_dv = (int)x.s_dv;
    if (args.segs > 1) {
      in = state_only ? nullptr : x.seg + (head * args.segs + order) * state_size;
      s_dk = x.DV; s_dv = 1;
    }
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)in, 0, in ? (int)state_size * 4 : 0, 0x00020000);
    const int dv = dv0 + 32 * w + (lane & 31);
#pragma unroll
    for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = 32 * (part * NDT + dt) + TK::state_row(i, lane);
        const uint32_t at = d < x.DK && dv < x.DV ? (uint32_t)(d * s_dk + dv * s_dv) * 4 : kNoRow;
        S[dt][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
      }
  }
  // fp16: S holds this lane's column of the state times a power of two; a bound
  // of its values, so that they stay below 2^100 with it: the power follows V, and
  // steps that have nearly died away would raise it past what fp32 holds
  float lift = 1.f, bound = 0.f;

  // Weights of P (row j = reg_row, column i = lane; times scale) and of V in the
  // state's sum (backwards times scale).  They count from the chunk's end forwards in time and from its
  // beginning backwards, so a chunk of fewer than 32 steps lies at that end of
  // its tiles.
  const int ri = lane & 31;
  const float scale = args.scale;
  float wp[16], wv[PB][EB];
  // (0 is for the rows that have no part in a step; what underflows is not)
  const float least = scale != 0.f ? 0x1p-149f : 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int j = reg_row(i, lane), e = rev ? j - ri : ri - j;
    const float x = decay.power(e < 0 ? 0 : e) * scale;
    wp[i] = e < 0 ? 0.f : x == 0.f ? least : x;
  }
#pragma unroll
  for (int pb = 0; pb < PB; ++pb)
#pragma unroll
    for (int e = 0; e < EB; ++e) {
      const int j = frag_row<T>(pb, e, lane);
      wv[pb][e] = decay.power(rev ? j + 1 : 31 - j) * (rev ? scale : 1.f);
    }
  const float keep32 = decay.power(32);
  const float rest32 = decay.beyond(32, keep32);  // of a^32
  float owed = 0.f;
  // forwards every row's power is the chunk's full one but in the last chunk
  const float since32 = decay.power(rev ? 31 - ri : ri + 1) * (rev ? 1.f : scale);
  // the state of this work-group reaches an output in fp32
  const bool state_out = x.s_out != nullptr && ha == 0;
  // (this wave's rows of the state: k-blocks from part KB of a, tiles from part NDT of k)
  static_assert(KB % 4 == 0 || KB == 2, "");
  const uint32_t row_first = KB % 4 == 0 ? TK::row_first(lane) + 128 * (part * KB / 4)
                                         : (TK::row_first(lane) ^ (64 * (part & 1))) + 128 * (part >> 1);
  uint32_t col_first = TK::col_first(lane, true);
  if constexpr (sizeof(T) == 4) col_first += 128 * part * NDT;
  else if constexpr (NDT % 2 == 0) col_first += 64 * part * NDT;
  else col_first = (col_first ^ (64 * (part & 1))) + 128 * (part >> 1);
  const uint32_t v_first = (TV::col_first(lane, false) + (sizeof(T) == 2 ? (w >> 1) * 128 : w * 128)) ^
                           (sizeof(T) == 2 ? (w & 1) * 64 : 0);  // columns 32 w ..
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void_t*)lds;

  // ---- loads: iteration it is chunk it / heads (in the order of time), head it % heads ----
  Rows32<T, DP, NW * KS, DMA> la, lk;
  Rows32<T, 32 * NW, NW * KS, DMA> lv;
  la.init(x.as.t, x.DK, x.whole & kWholeQ, wave, lane);
  lk.init(x.ks.t, x.DK, x.whole & kWholeK, wave, lane);
  lv.init(x.vs.t, cols < 32 * NW ? cols : 32 * NW, x.whole & kWholeV, wave, lane);
  const int64_t first_row = rev && n_chunks > 0 ? r0 + 32 * (int64_t)(n_chunks - 1) : r0, next = rev ? -32 : 32;
  const T* a0 = (const T*)x.a + b * x.as.b + ((int64_t)hs * x.ga + ha) * x.as.h + first_row * x.as.t;
  const T* k0 = (const T*)x.k + b * x.ks.b + (int64_t)hs * x.gb * x.ks.h + first_row * x.ks.t;
  const T* v0 = (const T*)x.v + b * x.vs.b + (int64_t)hs * x.gb * x.vs.h + first_row * x.vs.t + dv0;
  const int64_t a_head = KIND == kMany ? x.as.h : 0, k_head = KIND == kSum || state_only ? x.ks.h : 0,
                v_head = KIND == kSum || state_only ? x.vs.h : 0;
  // (32 rows of a tile that a descriptor reaches are below 2^30 bytes)
  typedef typename std::conditional<DMA, int, int64_t>::type step_t;
  const step_t a_next = (step_t)(next * x.as.t), k_next = (step_t)(next * x.ks.t), v_next = (step_t)(next * x.vs.t);
  constexpr int kLoadsA = state_only ? 0 : decltype(la)::kLoads, kLoadsKV = decltype(lk)::kLoads + decltype(lv)::kLoads;
  int left = steps, lh = 0;  // of the next load: steps not loaded yet, head
  uint32_t l_at = lds0, l_kv = lds0 + LL::kAtPairs;
  // steps of a chunk with `left` to go (backwards the last one, of fewer, is the first)
  auto chunk_steps = [&](int left) __attribute__((always_inline)) { return rev ? ((left - 1) & 31) + 1 : left < 32 ? left : 32; };
  auto load = [&]() __attribute__((always_inline)) {
    const int rows = chunk_steps(left), shift = rev ? 0 : 32 - rows;
    const uint32_t kv = KIND == kMany ? l_kv : l_at + LL::kA;
    const bool sum = KIND == kSum || state_only, pair = KIND != kMany || lh == 0;
    auto each = [&](auto full) __attribute__((always_inline)) {
      constexpr bool kFull = decltype(full)::value;
      if constexpr (!state_only) la.template load<kFull>(KIND == kMany ? a0 + lh * a_head : a0, rows, shift, l_at);
      if (pair) {
        lk.template load<kFull>(sum ? k0 + lh * k_head : k0, rows, shift, kv);
        lv.template load<kFull>(sum ? v0 + lh * v_head : v0, rows, shift, kv + TK::kBytes32);
      }
    };
    if (DMA && rows == 32) each(std::true_type{});
    else each(std::false_type{});
    if (KIND == kMany && pair) l_kv = l_kv == lds0 + LL::kAtPairs ? l_kv + LL::kKV : lds0 + LL::kAtPairs;
    l_at = l_at == lds0 + (NST - 1) * LL::kStage ? lds0 : l_at + LL::kStage;
    if (KIND == kOne || ++lh == heads) {
      lh = 0;
      left -= rows;
      a0 += a_next;
      k0 += k_next;
      v0 += v_next;
    }
  };

  // ---- stores ----
  constexpr int kKeep = kSplit ? 16 / KS : 16;  // registers of O that this wave stores
  constexpr int kGive = 256 * kKeep, kPassed = NW * KS * (KS - 1) * kGive;  // bytes for another wave, of all waves
  float keep_o[kKeep];
  T* out = (T*)x.out + b * x.os.b + ((int64_t)hs * x.ga + ha) * x.os.h + dv0 + 32 * w + (kSplit ? 32 / KS * part : 0) +
           (first_row + ri) * x.os.t;
  const int64_t o_row = x.os.t, o_next = next * o_row;
  int sh = 0;  // head of the next store
  const int out_cols = cols - 32 * w - (kSplit ? 32 / KS * part : 0);  // (may be below 0: no columns)
  const bool whole_o = (x.whole & kWholeO) && out_cols >= 2 * kKeep;
  uint32_t pass = lds0 + LL::kAtPass;
  // O of the iteration before, a chunk of n steps, to where `out` stands
  auto store = [&](int n) __attribute__((always_inline)) {
    const bool there = rev ? ri < n : ri >= 32 - n;
    T* p = n < 32 && !rev ? out - (32 - n) * o_row : out;
    if constexpr (KIND == kMany) p += sh * x.os.h;
    if constexpr (kSplit) {
      const uint32_t at = pass + wave * (KS - 1) * kGive + lane * 16;
#pragma unroll
      for (int i = 0; i < (KS - 1) * kKeep / 4; ++i) {
        float y[4];
        unpack<float>(*(lds_vec_t*)(uintptr_t)(at + i * 1024), y);
#pragma unroll
        for (int j = 0; j < 4; ++j) keep_o[4 * (i % (kKeep / 4)) + j] += y[j];
      }
      pass = pass == lds0 + LL::kAtPass ? pass + kPassed : lds0 + LL::kAtPass;
    }
    if (whole_o) {
      if constexpr (sizeof(T) == 2) {
        static_assert(kKeep % 8 == 0, "whole chunks of 16 bytes (KS = 4 is fp32's)");
        u32x4_t q[kKeep / 8];
#pragma unroll
        for (int i = 0; i < kKeep / 8; ++i) {
          const float* o = keep_o + 8 * i;
          const auto s0 = __builtin_amdgcn_permlane32_swap(pack2<T>(o[0], o[1]), pack2<T>(o[4], o[5]), false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(pack2<T>(o[2], o[3]), pack2<T>(o[6], o[7]), false, false);
          q[i] = u32x4_t{s0[0], s1[0], s0[1], s1[1]};
        }
        if (there) {
#pragma unroll
          for (int i = 0; i < kKeep / 8; ++i) *(u32x4_t*)(p + 16 * i + 8 * (lane >> 5)) = q[i];
        }
      } else if (there) {
#pragma unroll
        for (int i = 0; i < kKeep / 4; ++i) *(u32x4_t*)(p + reg_row(4 * i, lane)) = pack<float>(keep_o + 4 * i);
      }
    } else if (there) {
#pragma unroll 1
      for (int i = 0; i < kKeep; ++i) {
        float o = 0.f;  // (registers cannot be indexed: a loop keeps this rare path small)
#pragma unroll
        for (int j = 0; j < kKeep; ++j) o = j == i ? keep_o[j] : o;
        const int d = reg_row(i, lane);
        if (d < out_cols) p[d] = Elem<T>::from_f(o);
      }
    }
    if (KIND != kMany || ++sh == heads) {
      sh = 0;
      out += o_next;
    }
  };
  // O is complete: what this wave stores stays, the rest goes to the other
  // waves of its columns
  auto hand_over = [&](const f32x16_t& O) __attribute__((always_inline)) {
    if constexpr (kSplit) {
#pragma unroll
      for (int p = 0; p < KS; ++p) {
        if (p == part) {
#pragma unroll
          for (int i = 0; i < kKeep; ++i) keep_o[i] = O[kKeep * p + i];
        } else {
          // (of KS - 1 places of wave (w, p), the one for its part's distance)
          const uint32_t at = pass + ((w + NW * p) * (KS - 1) + ((part - p + KS) % KS - 1)) * kGive + lane * 16;
          float give[kKeep];
#pragma unroll
          for (int i = 0; i < kKeep; ++i) give[i] = O[kKeep * p + i];
#pragma unroll
          for (int i = 0; i < kKeep / 4; ++i) *(lds_vec_t*)(uintptr_t)(at + i * 1024) = pack<float>(give + 4 * i);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) keep_o[i] = O[i];
    }
  };

  const int iters = n_chunks * heads;
#pragma unroll
  for (int i = 0; i < NST - 1; ++i)
    if (i < iters) load();
  // The state is here: a wait left to its first use would stand in the loop, and
  // there wait for every chunk's loads (8 sequences, 16 heads of 128, 4096 steps,
  // bf16, forward: 266 us, so 229).
#pragma unroll
  for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+v"(S[dt][i]));
  auto most_of_state = [&]() __attribute__((always_inline)) {
    float most = 0.f;
#pragma unroll
    for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(S[dt][i]));
    return most;
  };
  if constexpr (kHalf && !state_only) {
#pragma unroll
    for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x = fabsf(S[dt][i]);
        bound = fmaxf(bound, x < INFINITY ? x : 0.f);
      }
  }

  f32x16_t O = zero16();
  float s_by = 1.f, undo = 1.f;       // fp16: of the state as an operand, and back
  u32x4_t s_op[KIND == kMany ? KB : 1];
  // the state as the operand of k-block kb
  auto state_operand = [&](int kb) __attribute__((always_inline)) {
    constexpr int kPer = sizeof(T) == 2 ? 2 : 4;  // k-blocks of a tile of the state
    if constexpr (kHalf) {
      f32x16_t s;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[8 * (kb % kPer) + i] = S[kb / kPer][8 * (kb % kPer) + i] * s_by;
      return TK::reg_frag(s, kb % kPer);
    } else {
      return TK::reg_frag(S[kb / kPer], kb % kPer);
    }
  };
  int togo = steps, g = 0, n_before = 0;
  uint32_t u_at = lds0, u_kv = lds0 + LL::kAtPairs;
  for (int it = 0; it < iters; ++it) {
    const bool first = KIND == kOne || g == 0, last = KIND == kOne || g == heads - 1;
    // this iteration's rows have come; those of the next (three stages) may be on their way
    if (NST == 2 || it + 1 >= iters) stage_barrier<0>();
    else if (KIND == kMany && !last) stage_barrier<kLoadsA>();
    else stage_barrier<kLoadsA + kLoadsKV>();
    if (!state_only && it > 0 && (KIND != kSum || first)) {
      store(n_before);
    }
    if (it + NST - 1 < iters) load();
    const uint32_t kv = KIND == kMany ? u_kv : u_at + LL::kA;
    const uint32_t rows_at = u_at + row_first, keys_at = kv + row_first, cols_at = kv + col_first,
                   v_at = kv + TK::kBytes32 + v_first;
    const int n = chunk_steps(togo);

    // V weighted for the state's sum, in 16 bits as two numbers (fp16 to 2^-22,
    // bf16 to 2^-17) and in bf16 as a third where the state is an fp32 output;
    // done between the products of the rows, which it covers
    constexpr int kParts = sizeof(T) == 4 ? 1 : kHalf ? 2 : 3;
    u32x4_t vf[PB], vw[PB][kParts];
    float un = 1.f;  // fp16: O's factor (of this lane's row) before it is complete
    float most_v = 0.f, vx[kHalf ? PB : 1][EB];
    const bool update = KIND != kMany || last;
    auto split = [&](int pb, float* f) __attribute__((always_inline)) {
      vw[pb][0] = pack<T>(f);
#pragma unroll
      for (int i = 1; i < kParts; ++i) {  // what the number before has rounded away
        if (i == 2 && !state_out) break;
        float r[EB];
        unpack<T>(vw[pb][i - 1], r);
#pragma unroll
        for (int e = 0; e < EB; ++e) f[e] -= r[e];
        vw[pb][i] = pack<T>(f);
      }
    };
    auto weigh = [&](int pb) __attribute__((always_inline)) {
      if (!update) return;
      float f[EB];
      unpack<T>(vf[pb], f);
#pragma unroll
      for (int e = 0; e < EB; ++e) f[e] *= wv[pb][e];
      if constexpr (kHalf) {
#pragma unroll
        for (int e = 0; e < EB; ++e) {
          vx[pb][e] = f[e];
          most_v = fmaxf(most_v, fabsf(f[e]));
        }
      } else {
        split(pb, f);
      }
    };
    auto read_v = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int pb = 0; pb < PB; ++pb) vf[pb] = TV::col_at(v_at, TK::KR * pb, 0);
    };

    if constexpr (state_only) {
      read_v();
#pragma unroll
      for (int pb = 0; pb < PB; ++pb) weigh(pb);
    } else {
      f32x16_t P = zero16();
      float zeros = 0.f;  // NaN where a value of V is not finite
      // fragments of V are weighed after the products of these k-blocks
      auto weigh_at = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int pb = 0; pb < PB; ++pb)
          if (kb == ((pb + 1) * KB + PB - 1) / PB - 1) {
            weigh(pb);
            zeros = add_zeros<T>(vf[pb], zeros);
          }
      };
      // rows of a and k in turn, k-block by k-block
      u32x4_t af;
      // (fewer where the registers are full: 64 sequences, 16 heads of 64, 256 steps,
      // bf16, backward 80 us with six ahead, 66 with four, 64 with three)
      constexpr int kFewer = DP == 64 && KS == 1 && KIND == kOne ? 3 : NDT * sizeof(T) >= 8 && KIND != kOne ? 2 : 0;
      Ahead<2 * KB, kAheadRows - kFewer> rows;
      auto read_rows = [&](int f) __attribute__((always_inline)) { return TK::row_at(f & 1 ? keys_at : rows_at, f >> 1); };
      if (KIND != kSum || first) {
        if constexpr (kHalf) {
          if (first) {
            const float down = inverse(lift), most = most_of_state() * down;
            // (a column that is not finite gives no number anyway)
            const float by = power_of_two(__builtin_amdgcn_readfirstlane(lift_bits(wave_max(most < INFINITY ? most : 0.f), -126, 60)));
            s_by = by * down;
            undo = inverse(by);
          }
        }
        if constexpr (KIND == kMany) {  // kept over the chunk's heads
          if (first) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) s_op[kb] = state_operand(kb);
          }
        }
        O = zero16();
        rows.start(read_rows);
        read_v();
        rows.run(read_rows, [&](int f, u32x4_t q) __attribute__((always_inline)) {
          const int kb = f >> 1;
          if (!(f & 1)) {
            af = q;
            return;
          }
          const u32x4_t sf = KIND == kMany ? s_op[kb] : state_operand(kb);
          P = Mm<T>::mac(q, af, P);
          O = Mm<T>::mac(sf, af, O);
          weigh_at(kb);
        });
        float f = since32;
        if (n < 32) {
          const int e = rev ? n - 1 - ri : ri + 1 - (32 - n);
          f = decay.power(e < 0 ? 0 : e) * (rev ? 1.f : scale);
        }
        if constexpr (kHalf) f *= undo;
#pragma unroll
        for (int i = 0; i < 16; ++i) O[i] *= f;
      } else {
        rows.start(read_rows);
        read_v();
        rows.run(read_rows, [&](int f, u32x4_t q) __attribute__((always_inline)) {
          if (!(f & 1)) {
            af = q;
            return;
          }
          P = Mm<T>::mac(q, af, P);
          weigh_at(f >> 1);
        });
      }
      // Values of V that are not finite would reach, times zero, the rows that
      // have no part in their steps: they are taken out, and their columns become
      // NaN from their step on.  (Forward and backward of 8 sequences, 16 heads of
      // 128, us: 4096 steps of bf16 168 and 354, with it 173 and 358; 2048 of fp32
      // 273 and 809, with it 279 and 830.)
      const bool odd = __any(zeros != 0.f);
      int edge = rev ? -1 : 32;
      if (__builtin_expect(odd, 0)) {  // (nothing of it is kept in registers over the chunks)
        const int ln = tile_lane<true>(lane);
#pragma unroll
        for (int pb = 0; pb < PB; ++pb) vf[pb] = finite_only<T>(vf[pb], pb, ln, rev, &edge);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) P[i] = mul_zero(P[i], wp[i]);
      float by = 1.f;
      if constexpr (kHalf) {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(P[i]));
        by = power_of_two(lift_bits(fmaxf(most, other_half(most)), -126, 40));  // (O times it stays in range)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          P[i] *= by;
          O[i] *= by;
        }
      }
#pragma unroll
      for (int pb = 0; pb < PB; ++pb) O = Mm<T>::mac(vf[pb], TK::reg_frag(P, pb), O);
      if (__builtin_expect(odd, 0)) {
        const int ln = tile_lane<true>(lane), row = ln & 31, other = __shfl(edge, ln ^ 32);
        edge = rev ? (other > edge ? other : edge) : (other < edge ? other : edge);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = __shfl(edge, reg_row(i, ln));
          if (rev ? row <= at : row >= at) O[i] = NAN;
        }
      }
      if constexpr (kHalf) un = inverse(by);
    }

    if (update) {
      float keep = (KIND == kSum || state_only) && !first ? 1.f : n < 32 ? decay.power(n) : keep32;
      // What a^32 is rounded by is made up for by its neighbours now and then, so
      // that it does not add up (65536 steps of memories of 20000 and more: the state
      // 2.8e-5 off, so 3e-6; in 16 bits the matrix cores' own sums are off by more).
      if (sizeof(T) == 4 && n == 32 && ((KIND != kSum && !state_only) || first)) {
        owed += rest32;
        keep = keep32 + owed;
        owed -= keep - keep32;
      }
      if constexpr (kHalf) {
        const float most = fmaxf(most_v, other_half(most_v));
        bound = bound * keep + most * 0x1p21f;  // (32 steps, keys up to 65504)
        const int cap = 354 - (int)(__float_as_uint(bound) >> 23), r = (int)lift_bits(most, -36, 90);
        const float to = power_of_two((uint32_t)(r < cap ? r : cap));  // (of 2^100 / bound, 2^-28 and more)
        keep *= to * inverse(lift);
        lift = to;
#pragma unroll
        for (int pb = 0; pb < PB; ++pb) {
#pragma unroll
          for (int e = 0; e < EB; ++e) vx[pb][e] *= to;
          split(pb, vx[pb]);
        }
      }
#pragma unroll
      for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) S[dt][i] *= keep;
      Ahead<PB * NDT, kAheadCols> kcols;
      auto read_cols = [&](int i) __attribute__((always_inline)) { return TK::col_at(cols_at, TK::KR * (i / NDT), i % NDT); };
      kcols.start(read_cols);
      kcols.run(read_cols, [&](int i, u32x4_t kf) __attribute__((always_inline)) {
        f32x16_t& s = S[i % NDT];
        s = Mm<T>::mac(kf, vw[i / NDT][0], s);
        if constexpr (kParts > 1) s = Mm<T>::mac(kf, vw[i / NDT][1], s);
        if constexpr (kParts > 2)
          if (state_out) s = Mm<T>::mac(kf, vw[i / NDT][2], s);
      });
    }
    // (last, when the products are done: the state's cover them)
    if constexpr (!state_only) {
      if constexpr (kHalf) {
#pragma unroll
        for (int i = 0; i < 16; ++i) O[i] *= un;
      }
      if (KIND != kSum || last) hand_over(O);
    }
    n_before = n;
    u_at = u_at == lds0 + (NST - 1) * LL::kStage ? lds0 : u_at + LL::kStage;
    if (last) {
      g = 0;
      togo -= n;
      if constexpr (KIND == kMany) u_kv = u_kv == lds0 + LL::kAtPairs ? u_kv + LL::kKV : lds0 + LL::kAtPairs;
    } else {
      ++g;
    }
  }
  if constexpr (!state_only) {
    if (iters > 0) {
      if constexpr (kSplit) stage_barrier<0>();
      store(n_before);
    }
    // steps past the end
    const int64_t top = r0 + args.seg_rows < args.T ? r0 + args.seg_rows : args.T;
    T* p0 = (T*)x.out + b * x.os.b + ((int64_t)hs * x.ga + ha) * x.os.h + dv0;
    constexpr int kChunks = 32 * NW / EB, kRows = 64 * NW * KS / kChunks;  // of 16 bytes a row, rows at a time
    const bool chunks = (x.whole & kWholeO) != 0;
    const int tid = wave * 64 + tile_lane<true>(lane), c = tid % kChunks * EB;
    for (int64_t row = r1 + tid / kChunks; row < top; row += kRows)
      for (int k = 0; k < (KIND == kMany ? x.ga : 1); ++k) {
        T* p = p0 + k * x.os.h + row * x.os.t + c;
        if (chunks) {
          if (c < cols) *(u32x4_t*)p = u32x4_t{0, 0, 0, 0};
        } else {
          for (int d = 0; d < EB && c + d < cols; ++d) p[d] = Elem<T>::from_f(0.f);
        }
      }
  }
  // the state after the run, or the segment's own sum
  float* to = nullptr;
  int s_dk = (int)x.s_dk, s_dv = (int)x.s_dv;
  if (state_only) {
    to = x.seg + (head * args.segs + order) * state_size;
    s_dk = x.DV; s_dv = 1;
  } else if (state_out && order == args.segs - 1) {
    to = x.s_out + head * state_size;
  }
  if (to) {
    const float by = inverse(lift);
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)to, 0, (int)state_size * 4, 0x00020000);
    const int ln = tile_lane<true>(lane), dv = dv0 + 32 * w + (ln & 31);
#pragma unroll
    for (int dt = 0; dt < NDT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = 32 * (part * NDT + dt) + TK::state_row(i, ln);
        const uint32_t at = d < x.DK && dv < x.DV ? (uint32_t)(d * s_dk + dv * s_dv) * 4 : kNoRow;
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(kHalf ? S[dt][i] * by : S[dt][i]), r, at, 0, 0);
      }
  }
}

template <typename T, int DP, int NW, int KS, bool DMA, int KIND>
static hipError_t linattn_launch(const LinArgs& a, unsigned groups, hipStream_t s) {
  constexpr size_t bytes = LinLds<T, DP, NW, KS, KIND>::kBytes;
  const hipError_t e = allow_lds<linattn_kernel<T, DP, NW, KS, DMA, KIND>>(bytes);
  if (e != hipSuccess) return e;
  Timed timed(10, s);
  linattn_kernel<T, DP, NW, KS, DMA, KIND><<<dim3(groups), 64 * NW * KS, bytes, s>>>(a);
  return hipGetLastError();
}
template <typename T, int DP, int NW, int KS, bool DMA>
static hipError_t linattn_kind(const LinArgs& a, int many, unsigned groups, hipStream_t s) {
  if (a.state_only) return linattn_launch<T, DP, NW, KS, DMA, kState>(a, groups, s);
  // (kSum does runs of kOne too)
  for (int i = 0; i < a.runs; ++i)
    if (a.run[i].gb > 1) return linattn_launch<T, DP, NW, KS, DMA, kSum>(a, groups, s);
  if (many) return linattn_launch<T, DP, NW, KS, DMA, kMany>(a, groups, s);
  return linattn_launch<T, DP, NW, KS, DMA, kOne>(a, groups, s);
}
template <typename T, int DP, int NW, int KS>
static hipError_t linattn_loads(const LinArgs& a, int many, int dma, unsigned groups, hipStream_t s) {
  return dma ? linattn_kind<T, DP, NW, KS, true>(a, many, groups, s) : linattn_kind<T, DP, NW, KS, false>(a, many, groups, s);
}
template <typename T>
static hipError_t linattn_of(const LinArgs& a, const LinTile& t, int many, int dma, unsigned groups, hipStream_t s) {
  switch (t.dp * 100 + t.nw * 10 + t.ks) {
    case 64 * 100 + 22: return linattn_loads<T, 64, 2, 2>(a, many, dma, groups, s);
    case 128 * 100 + 22: return linattn_loads<T, 128, 2, 2>(a, many, dma, groups, s);
    case 256 * 100 + 22: return linattn_loads<T, 256, 2, 2>(a, many, dma, groups, s);
    default: break;
  }
  if constexpr (sizeof(T) == 2) {
    if (t.dp == 64) return linattn_loads<T, 64, 2, 1>(a, many, dma, groups, s);
    if (t.dp == 128) return linattn_loads<T, 128, 4, 1>(a, many, dma, groups, s);
    return linattn_loads<T, 256, 4, 2>(a, many, dma, groups, s);
  } else {
    return linattn_loads<T, 128, 1, 4>(a, many, dma, groups, s);
  }
}

}  // namespace lstm
