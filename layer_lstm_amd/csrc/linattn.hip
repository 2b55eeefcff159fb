// linattn.hip -- linear attention: the plan, the launches by chunks, the join
// of a time axis cut into segments, and the kernel for a few steps (gfx950).
#include <type_traits>

#include "attend_common.hpp"
#include "model_internal.hpp"

namespace lstm {

void make_linattn_plan(const lstm_linattn_shape& s, int cus, LinPlan* p) {
  p->dtype = s.dtype;
  p->cus = cus;
  p->step = s.T <= LSTM_LINATTN_STEP;
  // Segments where the heads alone leave compute units idle: two work-groups a
  // unit, of four chunks at least.
  const int64_t heads = s.B * s.Hq * ((s.Dv + 127) / 128), chunks = (s.T + 31) / 32;
  int64_t segs = 1;
  if (heads > 0 && heads < cus) segs = 2 * (int64_t)cus / heads;
  if (segs > chunks / 4) segs = chunks / 4;
  if (segs < 1) segs = 1;
  p->seg_rows = (chunks + segs - 1) / segs * 32;
  if (p->seg_rows == 0) p->seg_rows = 32;
  p->segs = s.T > 0 ? (int)((s.T + p->seg_rows - 1) / p->seg_rows) : 1;
  p->seg_bytes = p->segs > 1 ? align256_seq((size_t)s.B * s.Hk * p->segs * s.D * s.Dv * 4) : 0;
  p->total_fwd = p->step ? 0 : p->seg_bytes;
  p->total_bwd = 3 * p->seg_bytes;
}

// The states at the segments' starts from the segments' own sums, in place:
// a thread an element, in the order of the run's time.
__global__ void __launch_bounds__(256) linattn_scan_kernel(LinArgs args) {
  const int which = blockIdx.z;
  const LinRun& x = args.run[which];
  const int n = x.DK * x.DV, e = blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  const int64_t head = blockIdx.y;
  const int b = (int)(head / args.Hs), hs = (int)(head - (int64_t)b * args.Hs);
  int64_t end = args.T;
  if (args.len) {
    const int64_t l = args.len[b];
    end = l < 0 ? 0 : l < args.T ? l : args.T;
  }
  float ld2 = args.log_decay[hs];
  ld2 = (ld2 > 0.f ? 0.f : ld2) * kLog2e;
  const int d = e / x.DV, c = e - d * x.DV;
  float S = x.s_in ? x.s_in[head * n + d * x.s_dk + c * x.s_dv] * x.in_by : 0.f;
  float* at = x.seg + head * args.segs * n + e;
  for (int o = 0; o < args.segs; ++o) {
    const int64_t seg = x.rev ? args.segs - 1 - o : o, r0 = seg * args.seg_rows;
    int64_t rows = end - r0;
    rows = rows < 0 ? 0 : rows < args.seg_rows ? rows : args.seg_rows;
    const float own = o + 1 < args.segs ? at[(int64_t)o * n] : 0.f;
    at[(int64_t)o * n] = S;
    S = (rows == 0 ? S : S * __builtin_amdgcn_exp2f(ld2 * (float)rows)) + own;
  }
}

static int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

static hipError_t launch_runs(int dtype, const LinArgs& a, int dp, int nw, int dma, int64_t groups, hipStream_t s) {
  if (groups == 0) return hipSuccess;
  if (dtype == LSTM_F32) return launch_linattn_f32(a, dp, nw, dma, (unsigned)groups, s);
  if (dtype == LSTM_BF16) return launch_linattn_bf16(a, dp, nw, dma, (unsigned)groups, s);
  return launch_linattn_f16(a, dp, nw, dma, (unsigned)groups, s);
}

hipError_t launch_linattn(const LinPlan& p, LinArgs a, const int* dma, hipStream_t s) {
  a.segs = p.segs;
  a.seg_rows = p.seg_rows;
  // runs of one kernel share a launch
  for (int pass = p.segs > 1 ? 0 : 1; pass < 2; ++pass) {
    bool done[3] = {false, false, false};
    for (int i = 0; i < a.runs; ++i) {
      if (done[i]) continue;
      LinArgs l = a;
      l.runs = 0;
      l.state_only = pass == 0;
      l.segs_of_launch = pass == 0 ? p.segs - 1 : p.segs;
      const int dp = padded(a.run[i].DK), nw = a.run[i].DV <= 64 ? 2 : 4;
      int64_t groups = 0;
      for (int j = i; j < a.runs; ++j) {
        if (done[j] || padded(a.run[j].DK) != dp || (a.run[j].DV <= 64 ? 2 : 4) != nw || dma[j] != dma[i]) continue;
        done[j] = true;
        LinRun& r = l.run[l.runs++];
        r = a.run[j];
        r.dv_blocks = (r.DV + 32 * nw - 1) / (32 * nw);
        r.group0 = groups;
        groups += (int64_t)a.B * (pass == 0 ? a.Hs : r.Ha) * r.dv_blocks * l.segs_of_launch;
      }
      const hipError_t e = launch_runs(p.dtype, l, dp, nw, dma[i], groups, s);
      if (e != hipSuccess) return e;
    }
    if (pass == 0 && a.B > 0 && a.Hs > 0) {
      int most = 0;
      for (int i = 0; i < a.runs; ++i) most = a.run[i].DK * a.run[i].DV > most ? a.run[i].DK * a.run[i].DV : most;
      Timed timed(10, s);
      linattn_scan_kernel<<<dim3((most + 255) / 256, (unsigned)(a.B * a.Hs), a.runs), 256, 0, s>>>(a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// A few steps: the state in registers in fp32, read and written once, which is
// the bound.  A work-group has a (sequence, key head) and 4 CL columns of its
// state: CL lanes of four columns, the rows dealt to the 256 / CL lane groups.
template <typename T, int CL, int RPT>
__global__ void __launch_bounds__(256) linattn_step_kernel(LinArgs args) {
  constexpr int RG = 256 / CL;  // row groups
  constexpr int HB = 4;         // query heads at a time
  const LinRun& x = args.run[0];
  __shared__ float qs[HB][256], ks[256], vs[4 * CL];
  __shared__ f32x4_t part[HB][RG][CL];
  const int tid = threadIdx.x, cl = tid % CL, rg = tid / CL;
  const int dvb = (int)(blockIdx.x % (unsigned)x.dv_blocks);
  const int64_t head = blockIdx.x / (unsigned)x.dv_blocks;
  const int b = (int)(head / args.Hs), hs = (int)(head - (int64_t)b * args.Hs);
  const int dv0 = dvb * 4 * CL, c0 = dv0 + 4 * cl;
  const bool whole = x.DV % 4 == 0 && ((uintptr_t)x.s_in & 15) == 0 && ((uintptr_t)x.s_out & 15) == 0;
  int end = (int)args.T;
  if (args.len) {
    const int l = args.len[b];
    end = l < 0 ? 0 : l < end ? l : end;
  }
  const float decay = __builtin_amdgcn_exp2f([&] {
    const float ld = args.log_decay[hs];
    return (ld > 0.f ? 0.f : ld) * kLog2e;
  }());
  f32x4_t S[RPT];
  const float* in = x.s_in ? x.s_in + head * x.DK * x.DV : nullptr;
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int d = rg + RG * r;
    S[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (in && d < x.DK) {
      const float* p = in + d * x.DV + c0;
      if (whole) {
        if (c0 < x.DV) S[r] = *(const f32x4_t*)p;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c0 + j < x.DV) S[r][j] = p[j];
      }
    }
  }
  for (int t = 0; t < (int)args.T; ++t) {
    const bool real = t < end;
    if (real) {
      __syncthreads();  // the step before has read k and v
      if (tid < x.DK) ks[tid] = Elem<T>::load((const T*)x.k + t * x.ks.t + b * x.ks.b + hs * x.ks.h + tid);
      if (tid < 4 * CL) vs[tid] = dv0 + tid < x.DV ? Elem<T>::load((const T*)x.v + t * x.vs.t + b * x.vs.b + hs * x.vs.h + dv0 + tid) : 0.f;
    }
    for (int g0 = 0; g0 < x.ga; g0 += HB) {
      const int heads = x.ga - g0 < HB ? x.ga - g0 : HB;
      if (real) {
        if (g0 > 0) __syncthreads();  // the heads before have been read
        for (int i = tid; i < heads * x.DK; i += 256) {
          const int g = i / x.DK, d = i - g * x.DK;
          qs[g][d] = Elem<T>::load((const T*)x.a + t * x.as.t + b * x.as.b + (int64_t)(hs * x.ga + g0 + g) * x.as.h + d);
        }
        __syncthreads();
        f32x4_t acc[HB];
#pragma unroll
        for (int g = 0; g < HB; ++g) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        const f32x4_t v = *(const f32x4_t*)(vs + 4 * cl);
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
          const int d = rg + RG * r;
          if (d < x.DK) {
            if (g0 == 0) {
              const float k = ks[d];
#pragma unroll
              for (int j = 0; j < 4; ++j) S[r][j] = S[r][j] * decay + k * v[j];
            }
#pragma unroll
            for (int g = 0; g < HB; ++g)
              if (g < heads) {
                const float q = qs[g][d];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[g][j] += q * S[r][j];
              }
          }
        }
#pragma unroll
        for (int g = 0; g < HB; ++g)
          if (g < heads) part[g][rg][cl] = acc[g];
        __syncthreads();
      }
      for (int i = tid; i < heads * 4 * CL; i += 256) {
        const int g = i / (4 * CL), c = i - g * 4 * CL;
        if (dv0 + c < x.DV) {
          float o = 0.f;
          if (real) {
#pragma unroll 8
            for (int k = 0; k < RG; ++k) o += ((const float*)&part[g][k][0])[c];
          }
          ((T*)x.out)[t * x.os.t + b * x.os.b + (int64_t)(hs * x.ga + g0 + g) * x.os.h + dv0 + c] = Elem<T>::from_f(as_f32(o * args.scale));
        }
      }
    }
  }
  if (!x.s_out) return;
  float* to = x.s_out + head * x.DK * x.DV;
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int d = rg + RG * r;
    if (d < x.DK) {
      float* p = to + d * x.DV + c0;
      if (whole) {
        if (c0 < x.DV) *(f32x4_t*)p = S[r];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c0 + j < x.DV) p[j] = S[r][j];
      }
    }
  }
}

template <typename T, int CL>
static hipError_t step_rows(const LinArgs& a, unsigned groups, hipStream_t s) {
  constexpr int RG = 256 / CL;
  Timed timed(10, s);
  if (a.run[0].DK <= 64) linattn_step_kernel<T, CL, 64 / RG><<<dim3(groups), 256, 0, s>>>(a);
  else if (a.run[0].DK <= 128) linattn_step_kernel<T, CL, 128 / RG><<<dim3(groups), 256, 0, s>>>(a);
  else linattn_step_kernel<T, CL, 256 / RG><<<dim3(groups), 256, 0, s>>>(a);
  return hipGetLastError();
}
template <typename T>
static hipError_t step_of(const LinPlan& p, LinArgs a, hipStream_t s) {
  LinRun& x = a.run[0];
  // 32 columns a work-group where 128 leave compute units idle
  const int64_t heads = (int64_t)a.B * a.Hs;
  const bool wide = heads * ((x.DV + 127) / 128) >= 2 * (int64_t)p.cus;
  x.dv_blocks = wide ? (x.DV + 127) / 128 : (x.DV + 31) / 32;
  const int64_t groups = heads * x.dv_blocks;
  if (groups == 0) return hipSuccess;
  return wide ? step_rows<T, 32>(a, (unsigned)groups, s) : step_rows<T, 8>(a, (unsigned)groups, s);
}

hipError_t launch_linattn_step(const LinPlan& p, const LinArgs& a, hipStream_t s) {
  if (p.dtype == LSTM_F32) return step_of<float>(p, a, s);
  if (p.dtype == LSTM_BF16) return step_of<bf16_t>(p, a, s);
  return step_of<f16_t>(p, a, s);
}

}  // namespace lstm
