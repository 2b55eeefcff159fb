// adamw.hip -- the AdamW step over many tensors in one launch, states in 32 or
// 8 bits, and the gradients' norm (gfx950).
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   w = w (1 - lr wd) - rate m / (sqrt(v) root + eps)
//
// Memory is the bound: a value takes 28 bytes with fp32 states (fp32
// parameters, or 16-bit ones with their fp32 copy), 16 with 8-bit states, and
// some 60 vector instructions (46.9 M fp32 values: 242 us, 5.4 TB/s; 250 M bf16
// values with 8-bit states 800 us, 5.0 TB/s; the norm reads at 5.9).  The tensors' table is the kernel's argument
// (no copy to the device, so a graph can hold the launch), a work-group finds
// its tensor by one compare per lane.
//
// 8-bit states: a block of 256 values is 32 lanes of 8; its largest is a
// reduction over them in registers, so that the new state is quantised from
// registers and every byte is read and written once.  sqrt(v) is held in place
// of v: an e4m3 number spans 2^18, which as v is 2^36, and what the update
// divides by is the root.  Rounding it up to the smallest number keeps a small
// v from becoming a division by eps alone.
//
// No operation is contracted: each is rounded as the formula has it, so that
// every path (vector loads or single ones, either launch shape) gives the same
// bits.
#include "internal.hpp"
#include "model_internal.hpp"

namespace lstm {

struct AdamwEntry {
  void* param;
  const void* grad;
  float* master;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
  float shrink;    // 1 - lr weight_decay
  uint32_t vec;    // every tensor is 16-byte aligned
};
struct AdamwArgs {
  AdamwEntry t[kAdamwTensors];
  uint32_t first[kAdamwTensors];  // its first work-group
  int count;
  float b1, c1, b2, c2, eps, rate, root;
  const lstm_adamw_control* control;
};

// The tensor of this work-group: the last whose first group is not past it.
__device__ __forceinline__ int entry_of(const uint32_t* first, int count, int lane) {
  const bool in = lane < count && first[lane < count ? lane : 0] <= blockIdx.x;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(in)) - 1);
}

template <typename T, int E>
__device__ __forceinline__ void load_values(const T* p, int64_t i, int64_t n, bool vec, float* f) {
  constexpr int V = vec_of<T>();
  if (vec && i + E <= n) {
#pragma unroll
    for (int j = 0; j < E; j += V) {
      if constexpr (E >= V) {
        unpack<T>(__builtin_nontemporal_load((const u32x4_t*)(p + i + j)), f + j);
      } else {  // four 16-bit values
        const uint2 u = *(const uint2*)(p + i);
        f[0] = f_of_bits16<T>(u.x & 0xffffu); f[1] = f_of_bits16<T>(u.x >> 16);
        f[2] = f_of_bits16<T>(u.y & 0xffffu); f[3] = f_of_bits16<T>(u.y >> 16);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) f[j] = i + j < n ? Elem<T>::load(p + i + j) : 0.f;
  }
}
template <typename T, int E>
__device__ __forceinline__ void store_values(T* p, int64_t i, int64_t n, bool vec, const float* f) {
  constexpr int V = vec_of<T>();
  if (vec && i + E <= n) {
#pragma unroll
    for (int j = 0; j < E; j += V) {
      if constexpr (E >= V) {
        __builtin_nontemporal_store(pack<T>(f + j), (u32x4_t*)(p + i + j));
      } else {
        *(uint2*)(p + i) = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (i + j < n) p[i + j] = Elem<T>::from_f(f[j]);
  }
}

// The largest of 32 lanes' values (every lane of the half gets it).
template <int Ctl>
__device__ __forceinline__ float dpp_max(float v) {
  return fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(v), (int)__float_as_uint(v), Ctl,
                                                                        0xf, 0xf, false)));
}
__device__ __forceinline__ float block_max(float v) {
  v = dpp_max<0xB1>(v);   // quad_perm 1,0,3,2
  v = dpp_max<0x4E>(v);   // quad_perm 2,3,0,1
  v = dpp_max<0x124>(v);  // row_ror:4
  v = dpp_max<0x128>(v);  // row_ror:8
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));  // the row of 16 beside it
}

constexpr float kLeast = 0x1p-100f;  // blocks of nothing above it are zeros
constexpr float kMost8 = 448.f, kLeast8 = 0x1p-9f;

// Eight values of a block as e4m3 numbers, and the block's scale.
template <bool Root>
__device__ __forceinline__ uint2 to_8bit(const float* x, float* scale) {
  float most = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[j]));
  most = block_max(most);
  const bool some = most > kLeast;
  *scale = some ? most * (1.f / kMost8) : 0.f;
  const float inv = some ? (1.f / most) * kMost8 : 0.f;
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = x[j] * inv;
    if (Root) y[j] = some && x[j] > 0.f && !(y[j] > kLeast8) ? kLeast8 : y[j];
    y[j] = y[j] > kMost8 ? kMost8 : y[j] < -kMost8 ? -kMost8 : y[j];  // (NaN stays)
  }
  uint2 u;
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  u.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  u.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], w, true);
  return u;
}
__device__ __forceinline__ void from_8bit(uint2 u, float scale, float* f) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = (int)(h ? u.y : u.x);
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    f[4 * h] = lo[0] * scale; f[4 * h + 1] = lo[1] * scale;
    f[4 * h + 2] = hi[0] * scale; f[4 * h + 3] = hi[1] * scale;
  }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int64_t i, int64_t n, bool vec) {
  if (vec && i + 8 <= n) return *(const uint2*)(p + i);
  uint2 u = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t c = i + j < n ? p[i + j] : 0;
    if (j < 4) u.x |= c << (8 * j);
    else u.y |= c << (8 * (j - 4));
  }
  return u;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, bool vec, uint2 u) {
  if (vec && i + 8 <= n) {
    *(uint2*)(p + i) = u;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) p[i + j] = (uint8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3)));
}

// Values of a lane: 16 bytes of fp32 states, 8 bytes of 8-bit ones.
template <int BITS> constexpr int lane_values() { return BITS == 8 ? 8 : 4; }

template <typename T, int BITS, int ROUNDS>
__global__ void __launch_bounds__(256) adamw_kernel(AdamwArgs a) {
#pragma clang fp contract(off)
  constexpr int E = lane_values<BITS>();
  float scale = 1.f, rate = a.rate, root = a.root;
  if (a.control) {
    if (a.control->skip) return;
    scale = a.control->scale;
    rate = a.control->rate;
    root = a.control->root;
  }
  const int lane = threadIdx.x & 63;
  const int k = entry_of(a.first, a.count, lane);
  const AdamwEntry& e = a.t[k];
  const uint32_t first = a.first[k];
  const int64_t base = (int64_t)(blockIdx.x - first) * (256 * E * ROUNDS);
  const bool vec = e.vec != 0;
  const float shrink = e.shrink;
  const int64_t n = e.n;
#pragma unroll 1
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t i = base + (int64_t)r * 256 * E + threadIdx.x * E;
    if (i - (BITS == 8 ? (threadIdx.x & 31) * E : 0) >= n) return;  // (8 bits: the lanes of a block stay together)
    float g[E], m[E], v[E], w[E];
    load_values<T, E>((const T*)e.grad, i, n, vec, g);
    if (e.master) load_values<float, E>(e.master, i, n, vec, w);
    else load_values<T, E>((const T*)e.param, i, n, vec, w);
    if constexpr (BITS == 8) {
      const int64_t blk = i >> 8;
      const uint2 mc = load_codes((const uint8_t*)e.m, i, n, vec), vc = load_codes((const uint8_t*)e.v, i, n, vec);
      from_8bit(mc, e.ms[blk], m);
      from_8bit(vc, e.vs[blk], v);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = v[j] * v[j];
    } else {
      load_values<float, E>((const float*)e.m, i, n, vec, m);
      load_values<float, E>((const float*)e.v, i, n, vec, v);
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float x = g[j] * scale;
      m[j] = m[j] * a.b1 + x * a.c1;
      v[j] = v[j] * a.b2 + (x * x) * a.c2;
      const float q = sqrtf(v[j]);
      w[j] = w[j] * shrink - (m[j] / (q * root + a.eps)) * rate;
      if (BITS == 8) v[j] = q;
    }
    if (e.master) store_values<float, E>(e.master, i, n, vec, w);
    store_values<T, E>((T*)e.param, i, n, vec, w);
    if constexpr (BITS == 8) {
      float sm, sv;
      const uint2 mc = to_8bit<false>(m, &sm), vc = to_8bit<true>(v, &sv);
      store_codes((uint8_t*)e.m, i, n, vec, mc);
      store_codes((uint8_t*)e.v, i, n, vec, vc);
      if ((threadIdx.x & 31) == 0) {
        e.ms[i >> 8] = sm;
        e.vs[i >> 8] = sv;
      }
    } else {
      store_values<float, E>((float*)e.m, i, n, vec, m);
      store_values<float, E>((float*)e.v, i, n, vec, v);
    }
  }
}

// ---- the gradients' norm ----
struct NormArgs {
  const void* grad[kAdamwTensors];
  int64_t n[kAdamwTensors];
  uint32_t vec[kAdamwTensors];
  uint32_t first[kAdamwTensors];
  int count;
  double* part;
};

// Sum over a work-group in a fixed order; thread 0 has it.
template <int W>
__device__ __forceinline__ double group_sum(double v) {
  __shared__ double sums[W];
  for (int d = 32; d > 0; d >>= 1) v += __shfl_down(v, d);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < W; ++i) s += sums[i];
  return s;
}

template <typename T>
__global__ void __launch_bounds__(256) adamw_norm_kernel(NormArgs a) {
  constexpr int E = vec_of<T>();
  const int k = entry_of(a.first, a.count, threadIdx.x & 63);
  const T* p = (const T*)a.grad[k];
  const int64_t n = a.n[k], lo = (int64_t)(blockIdx.x - a.first[k]) * kNormChunk;
  const int64_t hi = lo + kNormChunk < n ? lo + kNormChunk : n;
  double s = 0.0;
#pragma unroll 4
  for (int64_t i = lo + threadIdx.x * E; i < hi; i += 256 * E) {
    float f[E];
    load_values<T, E>(p, i, hi, a.vec[k] != 0, f);
#pragma unroll
    for (int j = 0; j < E; ++j) s = __builtin_fma((double)f[j], (double)f[j], s);
  }
  s = group_sum<4>(s);
  if (threadIdx.x == 0) a.part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(1024) adamw_control_kernel(const double* part, int64_t parts, double max_norm,
                                                             double unscale, double lr, double b1, double b2,
                                                             lstm_adamw_control* c) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < parts; i += 1024) s += part[i];
  s = group_sum<16>(s);
  if (threadIdx.x != 0) return;
  const double norm = unscale * sqrt(s);
  c->norm = (float)norm;
  const bool finite = norm <= 1.7976931348623157e308;
  c->skip = finite ? 0 : 1;
  if (!finite) return;
  const int64_t t = c->step + 1;
  c->step = t;
  c->scale = (float)(norm > max_norm ? unscale * (max_norm / norm) : unscale);
  c->rate = (float)(lr / (1.0 - pow(b1, (double)t)));
  c->root = (float)(1.0 / sqrt(1.0 - pow(b2, (double)t)));
}

// ---- launches ----
static bool entry_vec(const lstm_adamw_tensor& t) {
  return aligned16(t.param) && aligned16(t.grad) && aligned16(t.master) && aligned16(t.m) && aligned16(t.v);
}

template <typename T, int BITS, int ROUNDS>
static hipError_t step_launches(const AdamwPlan& p, const lstm_adamw_tensor* t, int64_t count,
                                const lstm_adamw_control* control, hipStream_t s) {
  constexpr int64_t kEach = 256 * lane_values<BITS>() * ROUNDS;
  AdamwArgs a;
  a.b1 = (float)p.b1; a.c1 = (float)(1.0 - p.b1);
  a.b2 = (float)p.b2; a.c2 = (float)(1.0 - p.b2);
  a.eps = (float)p.eps;
  a.rate = a.root = 0.f;
  if (!control) {
    a.rate = (float)(p.lr / (1.0 - __builtin_pow(p.b1, (double)p.step)));
    a.root = (float)(1.0 / __builtin_sqrt(1.0 - __builtin_pow(p.b2, (double)p.step)));
  }
  a.control = control;
  a.count = 0;
  int64_t groups = 0;
  auto launch = [&]() -> hipError_t {
    if (a.count == 0) return hipSuccess;
    Timed timed(12, s);
    adamw_kernel<T, BITS, ROUNDS><<<dim3((unsigned)groups), 256, 0, s>>>(a);
    a.count = 0;
    groups = 0;
    return hipGetLastError();
  };
  for (int64_t k = 0; k < count; ++k) {
    // a tensor of more work-groups than one launch has is several entries
    for (int64_t lo = 0; lo < t[k].n;) {
      const int64_t left = (t[k].n - lo + kEach - 1) / kEach;
      if (a.count == kAdamwTensors || groups == kMaxGroups) {
        const hipError_t e = launch();
        if (e != hipSuccess) return e;
      }
      const int64_t take = left < kMaxGroups - groups ? left : kMaxGroups - groups;
      AdamwEntry& x = a.t[a.count];
      const int64_t es = dtype_bytes(p.dtype), ss = BITS / 8;
      x.param = (char*)t[k].param + lo * es;
      x.grad = (const char*)t[k].grad + lo * es;
      x.master = t[k].master ? t[k].master + lo : nullptr;
      x.m = (char*)t[k].m + lo * ss;
      x.v = (char*)t[k].v + lo * ss;
      x.ms = BITS == 8 ? t[k].m_scale + lo / kAdamwBlock : nullptr;
      x.vs = BITS == 8 ? t[k].v_scale + lo / kAdamwBlock : nullptr;
      x.n = t[k].n - lo < take * kEach ? t[k].n - lo : take * kEach;
      x.shrink = (float)(1.0 - p.lr * t[k].weight_decay);
      x.vec = entry_vec(t[k]);
      a.first[a.count++] = (uint32_t)groups;
      groups += take;
      lo += x.n;
    }
  }
  return launch();
}

// A work-group takes four rounds of its lanes' loads where that leaves eight
// work-groups a compute unit, so that its start (the table, the control block)
// is paid once for them; fewer values are spread over more work-groups.
template <typename T, int BITS>
static hipError_t step_of(const AdamwPlan& p, const lstm_adamw_tensor* t, int64_t count,
                          const lstm_adamw_control* control, hipStream_t s) {
  int64_t n = 0;
  for (int64_t k = 0; k < count; ++k) n += t[k].n;
  int cus = 0;
  if (device_cus(&cus, nullptr) != LSTM_OK) return hipErrorInvalidDevice;
  return n >= (int64_t)cus * 8 * 4 * 256 * lane_values<BITS>() ? step_launches<T, BITS, 4>(p, t, count, control, s)
                                                               : step_launches<T, BITS, 1>(p, t, count, control, s);
}

template <typename T>
static hipError_t norm_launches(const lstm_adamw_tensor* t, int64_t count, double* part, int64_t* parts, hipStream_t s) {
  NormArgs a;
  a.count = 0;
  a.part = part;
  int64_t groups = 0;
  *parts = 0;
  auto launch = [&]() -> hipError_t {
    if (a.count == 0) return hipSuccess;
    Timed timed(12, s);
    adamw_norm_kernel<T><<<dim3((unsigned)groups), 256, 0, s>>>(a);
    a.part += groups;
    *parts += groups;
    a.count = 0;
    groups = 0;
    return hipGetLastError();
  };
  for (int64_t k = 0; k < count; ++k) {
    for (int64_t lo = 0; lo < t[k].n;) {
      const int64_t left = (t[k].n - lo + kNormChunk - 1) / kNormChunk;
      if (a.count == kAdamwTensors || groups == kMaxGroups) {
        const hipError_t e = launch();
        if (e != hipSuccess) return e;
      }
      const int64_t take = left < kMaxGroups - groups ? left : kMaxGroups - groups;
      a.grad[a.count] = (const T*)t[k].grad + lo;
      a.n[a.count] = t[k].n - lo < take * kNormChunk ? t[k].n - lo : take * kNormChunk;
      a.vec[a.count] = aligned16(t[k].grad);
      lo += a.n[a.count];
      a.first[a.count++] = (uint32_t)groups;
      groups += take;
    }
  }
  return launch();
}

hipError_t launch_adamw_step(const AdamwPlan& p, const lstm_adamw_tensor* t, int64_t count,
                             const lstm_adamw_control* control, hipStream_t s) {
  switch (p.dtype * 2 + (p.bits == 8)) {
    case 0: return step_of<float, 32>(p, t, count, control, s);
    case 1: return step_of<float, 8>(p, t, count, control, s);
    case 2: return step_of<bf16_t, 32>(p, t, count, control, s);
    case 3: return step_of<bf16_t, 8>(p, t, count, control, s);
    case 4: return step_of<f16_t, 32>(p, t, count, control, s);
    default: return step_of<f16_t, 8>(p, t, count, control, s);
  }
}

hipError_t launch_adamw_norm(const AdamwPlan& p, const lstm_adamw_tensor* t, int64_t count, double max_norm,
                             double unscale, double* ws, lstm_adamw_control* control, hipStream_t s) {
  int64_t parts = 0;
  const hipError_t e = p.dtype == LSTM_F32    ? norm_launches<float>(t, count, ws, &parts, s)
                       : p.dtype == LSTM_BF16 ? norm_launches<bf16_t>(t, count, ws, &parts, s)
                                              : norm_launches<f16_t>(t, count, ws, &parts, s);
  if (e != hipSuccess) return e;
  Timed timed(12, s);
  adamw_control_kernel<<<dim3(1), 1024, 0, s>>>(ws, parts, max_norm, unscale, p.lr, p.b1, p.b2, control);
  return hipGetLastError();
}

}  // namespace lstm
