// attend_common.hpp -- what the cross-attention kernels share: 32 x 32 MFMA
// fragments, tiles of rows in LDS, and the row addressing.
//
// Rows.  The query heads of one key head read the same keys, so for each
// (sequence b, key head) the kernels treat the M = Tq G queries of its
// G = Hq / Hk heads as rows r = t G + g of one matrix; shared heads need no
// other care, forward or backward.
//
// Tiles.  A tile holds N rows of DP values (D rounded up, the rest zeros) in
// 16-byte chunks; chunk c of row r sits at chunk r C + (c ^ swizzle(r)), C
// chunks a row, so that both ways of reading it spread over the LDS banks:
//   along the row (row_frag): lane l holds 16 bytes of row l % 32, the k
//     index along d;
//   across the rows (col_frag): lane l holds column l % 32, the k index along
//     the rows (16-bit types by ds_read_b64_tr_b16, fp32 by 4-byte reads).
//
// The product of two tiles leaves a 32 x 32 result with column l % 32 in lane
// l and rows 8 (i / 4) + 4 (l / 32) + i % 4 in register i.  Those registers
// are the other operand of the next product as they stand (rounded to the
// storage type, in fp32 not at all): a k index may be permuted as long as
// both operands agree, and col_frag reads the rows in that order.
#pragma once
#include <atomic>

#include "internal.hpp"
#include "seq_internal.hpp"

namespace lstm {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4_lds_t;
typedef __attribute__((address_space(3))) s16x4_lds_t lds_tr_t;

// One k-block of a 32 x 32 product: 16 bytes of each operand per lane.
//  16 bits: 16 k values, lane group l / 32 holding 8 of them;
//  fp32: 8 k values, lane group l / 32 holding 4 of them, one per MFMA.
template <typename T> struct Mm;
template <> struct Mm<bf16_t> {
  __device__ __forceinline__ static f32x16_t mac(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
};
template <> struct Mm<f16_t> {
  __device__ __forceinline__ static f32x16_t mac(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  }
};
template <> struct Mm<float> {
  __device__ __forceinline__ static f32x16_t mac(u32x4_t a, u32x4_t b, f32x16_t c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
};

template <typename T, int DP>
struct Tile {
  static constexpr int C = DP * (int)sizeof(T) / 16;    // chunks per row
  static constexpr int KB = C / 2;                      // k-blocks along d
  static constexpr int KR = sizeof(T) == 2 ? 16 : 8;    // rows of one k-block across the rows
  static constexpr int PB = 32 / KR;                    // k-blocks of 32 rows
  static constexpr int kBytes32 = 32 * C * 16;          // bytes of 32 rows
  static_assert(C % 4 == 0, "rows of whole 64 bytes");

  // Where C is a multiple of 8 (rows of whole 128 bytes) eight consecutive
  // rows take eight different chunks of 128 bytes, and four consecutive ones
  // both halves of it; else two rows lie 64 bytes apart already.
  __device__ __forceinline__ static int swizzle(int r) {
    return C % 8 == 0 ? ((r & 1) << 2) | ((r >> 1) & 3) : (r >> 1) & 3;
  }
  __device__ __forceinline__ static int chunk_at(int r, int c) { return (r * C + (c ^ swizzle(r))) * 16; }

  // rows row0 .. row0 + 31 (row0 a multiple of 8), k-block kb along d
  __device__ __forceinline__ static u32x4_t row_frag(const char* lds, int row0, int kb, int lane) {
    return *(const u32x4_t*)(lds + row0 * C * 16 + chunk_at(lane & 31, 2 * kb + (lane >> 5)));
  }
  // columns 32 dt .. 32 dt + 31, the KR rows from row0 (a multiple of 8)
  __device__ __forceinline__ static u32x4_t col_frag(const char* lds, int row0, int dt, int lane) {
    u32x4_t out;
    if constexpr (sizeof(T) == 2) {
      const int L = lane & 15, r = 4 * (lane >> 5) + (L >> 2);
      const int d = 32 * dt + 16 * ((lane >> 4) & 1) + 4 * (L & 3);
      const char* p = lds + row0 * C * 16 + chunk_at(r, d >> 3) + (d & 7) * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const s16x4_lds_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_t*)(p + h * 8 * C * 16));
        const uint2 u = __builtin_bit_cast(uint2, v);
        out[2 * h] = u.x;
        out[2 * h + 1] = u.y;
      }
    } else {
      const int d = 32 * dt + (lane & 31), g = lane >> 5;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        out[s] = *(const uint32_t*)(lds + row0 * C * 16 + chunk_at(4 * g + s, d >> 2) + (d & 3) * 4);
    }
    return out;
  }
  // the operand of rows KR pb .. from a product's registers
  __device__ __forceinline__ static u32x4_t reg_frag(const f32x16_t& s, int pb) {
    u32x4_t out;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = pack2<T>(s[8 * pb + 2 * i], s[8 * pb + 2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = __float_as_uint(s[4 * pb + i]);
    }
    return out;
  }
};

// F fragments read from LDS LA ahead of their products: start() issues the
// first LA reads, run() multiplies fragment f and issues the read of f + LA in
// its place.  The order is pinned (left alone, the compiler reads each
// fragment right before its product and waits for it).
template <int F, int LA_>
struct Ahead {
  static constexpr int LA = LA_ < F ? LA_ : F;
  u32x4_t buf[LA];
  template <class Read>
  __device__ __forceinline__ void start(Read read) {
#pragma unroll
    for (int f = 0; f < LA; ++f) buf[f] = read(f);
    __builtin_amdgcn_sched_barrier(0);
  }
  template <class Read, class Use>
  __device__ __forceinline__ void run(Read read, Use use) {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      use(f, buf[f % LA]);
      if (f + LA < F) buf[f % LA] = read(f + LA);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// The LDS addresses of a tile's fragments depend on the lane alone, and the
// compiler keeps them, some twenty registers, over all tiles.  Where a wave's
// rows fill the registers and spill, Lean computes them anew for each tile.
// Without / with it, 16 sequences, 16/8 heads, 512 x 512, us: backward bf16
// heads of 256 412 / 391, fp32 of 64 643 / 502, of 128 1876 / 1440, of 256
// 4080 / 2490; forward fp32 of 128 342 / 310, of 256 846 / 642.  Where nothing
// spills it costs: backward bf16 of 64 91 / 98, forward 35.7 / 37.0.
template <bool Lean>
__device__ __forceinline__ int tile_lane(int lane) {
  if constexpr (Lean) asm volatile("" : "+v"(lane));
  return lane;
}

__device__ __forceinline__ f32x16_t zero16() {
  f32x16_t z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}
// Row of a product's register i.
__device__ __forceinline__ int reg_row(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

// The value of lane l ^ 32.
__device__ __forceinline__ float other_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// 4 bytes per lane from a buffer straight into LDS, to lds + 4 * lane (see
// lds_dma16).
__device__ __forceinline__ void lds_dma4(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t voff) {
  const uint32_t m0v = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)lds);
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %1\n\tbuffer_load_dword %0, %2, 0 offen lds"
               :
               : "v"(voff), "s"(m0v), "s"(r)
               : "memory", "m0");
#pragma clang diagnostic pop
}

// 16 bytes of a row of D values from d: element by element where rows are
// not whole 16-byte chunks (values past D are zeros).
template <typename T>
__device__ __forceinline__ u32x4_t load_chunk(const T* row, int d, int D, bool whole) {
  constexpr int E = vec_of<T>();
  if (whole) {
    u32x4_t z = {0, 0, 0, 0};
    return d < D ? *(const u32x4_t*)(row + d) : z;
  }
  T e[E];
#pragma unroll
  for (int i = 0; i < E; ++i) e[i] = d + i < D ? row[d + i] : T(0);
  return __builtin_bit_cast(u32x4_t, e);
}

// What a call reads and writes; strides in elements.
struct AttendArgs {
  const void *q, *k, *v, *o, *dout;
  void *out, *dq, *dk, *dv;
  lstm_stride qs, ks, vs, os, gs, dqs, dks, dvs;  // gs: of dout
  float* lse;            // [B][Hq][Tq] (the backward reads it)
  float* stats;          // [B][Hq][Tq][2] backward: lse in powers of two (+inf: no key), sum_d dout o
  const int32_t* len;    // [B] or null
  const uint8_t* mask;   // [B][Tk] or null
  int64_t mask_b;
  int Tq, Tk, B, Hq, Hk, G, D;
  uint32_t M;            // Tq G rows of a (sequence, key head)
  float scale;
  int tiles, spread;     // work-groups per (sequence, key head); see group_of()
  int splits;            // parts of the keys (step kernel)
  float *part, *part_ml; // their outputs and (m, l)
  int whole;             // bits kWhole*: rows are whole aligned 16-byte chunks
};
constexpr int kWholeQ = 1, kWholeK = 2, kWholeV = 4, kWholeO = 8, kWholeG = 16, kWholeDq = 32, kWholeDk = 64,
              kWholeDv = 128;

// Work-group i of `tiles` per (sequence, key head): with `spread` unset the
// groups of eight pairs are dealt so that the tiles of one pair, which read
// the same rows, run on one XCD (work-groups go to the XCDs round robin) and
// share its L2 (64 pairs, 1024 x 2048, heads of 128: forward 76 us, dealt in
// order 97; of 64, 512 rows 36.5 and 36.7).  False: no work.
__device__ __forceinline__ bool group_of(const AttendArgs& a, uint32_t i, int* grp, int* tile) {
  const uint32_t n = (uint32_t)a.B * a.Hk;
  uint32_t g;
  if (a.spread) {
    g = i / a.tiles;
    *tile = (int)(i - g * a.tiles);
  } else {
    const uint32_t slot = i >> 3, s = slot / a.tiles;
    g = s * 8 + (i & 7);
    *tile = (int)(slot - s * a.tiles);
  }
  *grp = (int)g;
  return g < n;
}

// The grid of a.tiles work-groups per (sequence, key head).  Dealing the pairs
// in eights leaves XCDs idle where their number is small and odd.
static inline unsigned attend_grid(AttendArgs* a) {
  const unsigned n = (unsigned)a->B * (unsigned)a->Hk;
  a->spread = !(n % 8 == 0 || n >= 64);
  return (a->spread ? n : (n + 7) / 8 * 8) * (unsigned)a->tiles;
}
// Dynamic LDS past 64 KB has to be asked for, once per kernel (the static
// is the instance's own) and device.
template <auto Kernel>
static inline hipError_t allow_lds(size_t bytes) {
  if (bytes <= 64 * 1024) return hipSuccess;
  static std::atomic<uint64_t> asked{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (bit && (asked.load(std::memory_order_relaxed) & bit)) return hipSuccess;
  e = hipFuncSetAttribute((const void*)Kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == hipSuccess) asked.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Valid keys of a sequence: below its length (and not masked).
__device__ __forceinline__ int keys_of(const AttendArgs& a, int b) {
  if (!a.len) return a.Tk;
  const int n = a.len[b];
  return n < 0 ? 0 : n < a.Tk ? n : a.Tk;
}
// One bit per key of the 64 from key0.
__device__ __forceinline__ uint64_t key_bits(const uint8_t* mask, int key0, int end, int lane) {
  const int k = key0 + lane;
  bool ok = k < end;
  if (mask && ok) ok = mask[k] != 0;
  return __ballot(ok);
}

// Loads tiles of N consecutive rows (row r at p + r st) into LDS with NW
// waves: rows at or past `end`, rows of a zero mask byte and values past D
// become zeros.  DMA: straight into LDS (rows of whole 16-byte chunks, st >=
// D so that an offset of a row past `end` is past the descriptor's end, N st
// below 2^31 bytes); else chunk by chunk through registers.
constexpr uint32_t kNoRow = 0x80000000u;  // an offset past every descriptor's end

template <typename T, int DP, int N, int NW, bool DMA>
struct Loader {
  using TL = Tile<T, DP>;
  static constexpr int kTotal = N * TL::C / 64;            // loads of 1 KB of a tile
  static constexpr int kLoads = (kTotal + NW - 1) / NW;    // per wave, at most
  __device__ __forceinline__ bool mine(int j) const { return kTotal % NW == 0 || j * NW + w < kTotal; }
  const T* p;
  int64_t st;
  const uint8_t* mask;
  int D, whole, w, lane;
  // Byte offset of this lane's chunk of each load in the tile's rows.  Where
  // a load is whole rows, a multiple of the swizzle's eight, on from the one
  // before, one offset and the (uniform) step between them stand for all.
  static constexpr int kStepRows = 64 * NW % TL::C == 0 ? 64 * NW / TL::C : 0;
  static constexpr bool kStep = kStepRows > 0 && kStepRows % 8 == 0;
  uint32_t off[DMA && !kStep ? kLoads : 1];
  uint32_t step;

  __device__ __forceinline__ void init(const T* p_, int64_t st_, int D_, int whole_, const uint8_t* mask_, int w_,
                                       int lane_) {
    p = p_; st = st_; D = D_; whole = whole_; mask = mask_; w = w_; lane = lane_;
    step = (uint32_t)(kStepRows * (int)st * (int)sizeof(T));
    if constexpr (DMA) {
#pragma unroll
      for (int j = 0; j < (kStep ? 1 : kLoads); ++j) {
        const int i = (j * NW + w) * 64 + lane, r = i / TL::C, c = (i % TL::C) ^ TL::swizzle(r);
        off[j] = c * 16 < D * (int)sizeof(T) ? (uint32_t)(r * (int)st * (int)sizeof(T) + c * 16) : kNoRow;
      }
    }
  }
  __device__ __forceinline__ void load(int row0, int end, char* lds) const {
    if constexpr (DMA) {
      const int rows = end - row0 < N ? end - row0 : N;
      const int bytes = rows > 0 ? (int)(((rows - 1) * (int)st + D) * (int)sizeof(T)) : 0;
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc((void*)(p + (int64_t)row0 * st), 0, bytes, 0x00020000);
      uint32_t o[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        o[j] = kStep ? off[0] + j * step : off[j];  // (past every end stays past it)
        if (mask) {
          const int k = row0 + ((j * NW + w) * 64 + lane) / TL::C;
          if (mine(j) && (k >= end || mask[k] == 0)) o[j] = kNoRow;
        }
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        if (mine(j)) lds_dma16<false>(r, lds + (j * NW + w) * 1024, o[j], 0);
    } else {
      for (int j = 0; j < kLoads; ++j) {
        if (!mine(j)) break;
        const int i = (j * NW + w) * 64 + lane, r = i / TL::C, c = (i % TL::C) ^ TL::swizzle(r), k = row0 + r;
        u32x4_t v = {0, 0, 0, 0};
        if (k < end && (!mask || mask[k] != 0)) v = load_chunk<T>(p + (int64_t)k * st, c * vec_of<T>(), D, whole != 0);
        *(u32x4_t*)(lds + i * 16) = v;
      }
    }
  }
};

// The kernels for few rows or keys give every wave of a work-group its own
// tiles of the axis they sum over: as many waves (up to 8) as hold the two
// tiles of 32 rows they read in 128 KB; their loads overlap each other's
// products, and their sums are joined in LDS.
constexpr int step_waves_of(int64_t two_tiles) {
  return 128 * 1024 / two_tiles >= 8 ? 8 : 128 * 1024 / two_tiles >= 4 ? 4 : 2;
}
template <typename T, int DP> constexpr int step_waves() { return step_waves_of(2 * Tile<T, DP>::kBytes32); }

// Sum over the waves of their products' registers (column lane % 32), each in
// its own part (two tiles) of LDS; `f(d, v)` takes the sums of column
// lane % 32, whose rows d are dealt to the waves and the halves of a wave.
// Every wave has read its tiles when it calls this.
template <typename T, int DP, class F>
__device__ __forceinline__ void join_waves(const f32x16_t* acc, char* lds, int D, int w, int lane, F f) {
  constexpr int NW = step_waves<T, DP>(), kPart = 2 * Tile<T, DP>::kBytes32;
  static_assert(DP * 32 * 4 <= kPart, "a wave's registers fit its part");
  float* mine = (float*)(lds + w * kPart);  // [DP][32]
  __syncthreads();
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) mine[(32 * dt + reg_row(i, lane)) * 32 + (lane & 31)] = acc[dt][i];
  __syncthreads();
  for (int d = 2 * w + (lane >> 5); d < D; d += 2 * NW) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) v += ((const float*)(lds + k * kPart))[d * 32 + (lane & 31)];
    f(d, v);
  }
}

// 16-byte operands along d of one row in registers (zeros where !ok).
template <typename T, int DP>
__device__ __forceinline__ void load_row_frags(const T* row, int D, bool whole, bool ok, int lane, u32x4_t* f) {
  using TL = Tile<T, DP>;
#pragma unroll
  for (int kb = 0; kb < TL::KB; ++kb) {
    u32x4_t z = {0, 0, 0, 0};
    f[kb] = ok ? load_chunk<T>(row, (2 * kb + (lane >> 5)) * vec_of<T>(), D, whole) : z;
  }
}

// A row's column of products (register i of d-tile dt: d = 32 dt +
// reg_row(i)) times `by`, or zeros, to global memory.
template <typename T, int DP>
__device__ __forceinline__ void store_col(T* row, const f32x16_t* acc, float by, int D, bool whole, int lane,
                                          bool ok = true) {
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 32 * dt + reg_row(4 * i, lane);
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = ok ? as_f32(acc[dt][4 * i + j] * by) : 0.f;
      if (whole) {
        if (d < D) {
          if constexpr (sizeof(T) == 4) {
            *(f32x4_t*)(row + d) = f32x4_t{f[0], f[1], f[2], f[3]};
          } else {
            *(uint2*)(row + d) = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (d + j < D) row[d + j] = Elem<T>::from_f(f[j]);
      }
    }
}

}  // namespace lstm
