// linattn.hip -- linear attention: the plan, the launches by chunks, the join
// of a time axis cut into segments, and the kernel for a few steps (gfx950).
#include <type_traits>

#include "attend_common.hpp"
#include "linattn_decay.hpp"
#include "model_internal.hpp"

namespace lstm {

// The instance for rows of DK and DV values: `few` work-groups take the one of
// shorter iterations (two waves for 32 columns; fp32, bound by a wave's chain of
// matrix instructions, four, and the same instance for all runs, which then are
// one launch), which takes more work in all.
static LinTile linattn_tile(int64_t DK, int64_t DV, int dtype, bool few) {
  LinTile t;
  t.dp = DK <= 64 ? 64 : DK <= 128 ? 128 : 256;
  const bool f32 = dtype == LSTM_F32;
  if (f32 && few && t.dp <= 128) t = {128, 1, 4};
  else if (t.dp == 64) t = {64, 2, f32 || few ? 2 : 1};
  else if (t.dp == 128) t = f32 || few || DV <= 64 ? LinTile{128, 2, 2} : LinTile{128, 4, 1};
  else t = LinTile{256, f32 || DV <= 64 ? 2 : 4, 2};
  return t;
}

// How a call's runs are cut into work-groups.  The heads alone, where they fill
// the device: an iteration of a work-group is a chunk, and one work-group after
// the other reads its sequence once.  Else first by columns (two work-groups a
// head of more than 64), then the time axis into segments of four chunks at
// least, whose own sums a launch before has to find (k and v read twice).
// (8 sequences, 16 heads of 128, 4096 steps, bf16, forward, us: 128 work-groups
// 210, two a head 181, four segments 202; 2 sequences, 4 heads: 204, 159, 16
// segments of two a head 35, of one 42.)  Two segments cost what they gain (4
// sequences, 16 heads, 2048 steps: forward 82, in two 84, backward 115 and 152),
// and so do two work-groups a head that are more than the compute units (12
// sequences, 16 heads, 2048 steps, forward: 121, two a head 133; 8 sequences, 8
// heads, 1024 steps, fp16, backward: 73 and 88).  Where the segments have many
// chunks to go, whole heads (32768 steps, 32/8 heads, fp16: 223, two a head 284).
// Heads that share a state take one work-group (one update of the state for all
// of them) unless that leaves compute units idle (8 sequences, 6/3 heads of 80,
// 191 steps, fp32: 56 us, heads apart 32; 32 sequences, 32/8 heads, 1024 steps,
// fp16: 201, apart 255).  fp32's instance for few work-groups has a compute unit
// to itself: it is taken where all of them have one, and no run is long (forward
// and backward of the fp32 case above 83 us, so 65; 32 heads of 64, 8192 steps,
// cut into segments either way 466 and 900).
//   The numbers (bf16, heads of 128, forward and backward, us, where no other is
// named): work-groups of 64-value rows fill the device with two a compute unit (16
// sequences, 16 heads of 64, 1024 steps: 40 and 62, with one 47 and 62; 8
// sequences, 2048 steps: 57 and 93, with one 70 and 108).  Runs are long from 16
// chunks a compute unit on (2 sequences, 8 heads, 4096 steps: forwards, with 8, 51
// as they are, 57 as long ones; backwards, with 24, 80 as long ones and 101; 8192
// steps, with 16 and 48, 75 and 130, 84 and 179 as short ones).  A segment has four
// chunks at least (1 sequence, 8 heads, 512 steps: 23 and 29, two 21 and 33, eight
// 26 and 26; fp32 of 64 values 27 and 29, two 21 and 33, eight 49 and 50).  Segments
// make two work-groups a compute unit (1 sequence, 16 heads, 16384 steps: 109 and
// 250, one 122 and 292, three 121 and 261), forwards one where rows of 256 values
// fill it and where runs are short (1 sequence, 8 heads of 256, 8192 steps: 103,
// two 126; backwards, whose three runs do not end together, 260 and 240; fp32, 4096
// steps, 572 and 972; 1 sequence, 8 heads, 2048 steps, backwards: 42, one 46, fp32
// 110 and 181; 4 sequences, 16 heads of 64, 2048 steps, backwards: 67, three for
// two compute units 64, which 64-value rows take).
static void plan_call(const lstm_linattn_shape& s, int cus, int runs, const int64_t (*sizes)[3], LinCall* c) {
  const int64_t sets = s.B * s.Hk, chunks = (s.T + 31) / 32, most = chunks / 4 > 1 ? chunks / 4 : 1;
  bool fits = true;  // the device has a compute unit for all work-groups, or for the next when the short ones end
  auto groups = [&](bool few) {
    int64_t n = 0, iterations = 0, longest = 1;
    for (int i = 0; i < runs; ++i) {
      const int64_t DK = sizes[i][0], DV = sizes[i][1], ga = sizes[i][2];
      c->tile[i] = linattn_tile(DK, DV, s.dtype, few);
      const int64_t blocks = (DV + 32 * c->tile[i].nw - 1) / (32 * c->tile[i].nw);
      c->many[i] = ga > 1 && sets * blocks * most >= cus;
      const int64_t mine = sets * blocks * (c->many[i] ? 1 : ga), heads = i > 0 ? sizes[0][2] : c->many[i] ? ga : 1;
      n += mine;
      iterations += mine * heads;
      if (heads > longest) longest = heads;
    }
    fits = iterations <= cus * longest;
    return n;
  };
  int64_t n = groups(false), segs = 1;
  const bool small = c->tile[0].dp == 64;  // (work-groups of 64-value rows are half as large)
  const int64_t full = small ? 2 * (int64_t)cus : cus;
  if (n > 0 && n < full) {
    const bool long_runs = n * chunks >= 16 * (int64_t)cus;
    int64_t fine = groups(true);
    if (s.dtype == LSTM_F32 && (long_runs || !fits)) fine = groups(false);
    if (fine > full && !small && s.dtype != LSTM_F32) {
      n = groups(false);
    } else if (fine >= (small ? cus : full)) {
      n = fine;
    } else if (long_runs && !small) {
      n = groups(false);
      segs = (runs == 1 && c->tile[0].dp == 256 ? full : 2 * full) / n;
    } else {
      n = fine;
      const int64_t fill = c->tile[0].nw == 1 ? cus : full;
      segs = (runs == 1 ? fill : small ? 3 * fill / 2 : 2 * fill) / n;
    }
    if (segs > most) segs = most;
    if (segs < 3) segs = 1;
  }
  c->seg_rows = (chunks + segs - 1) / segs * 32;
  if (c->seg_rows == 0) c->seg_rows = 32;
  c->segs = s.T > 0 ? (int)((s.T + c->seg_rows - 1) / c->seg_rows) : 1;
}

void make_linattn_plan(const lstm_linattn_shape& s, int cus, LinPlan* p) {
  p->dtype = s.dtype;
  p->cus = cus;
  p->step = s.T <= LSTM_LINATTN_STEP;
  const int64_t G = s.Hk > 0 ? s.Hq / s.Hk : 1;
  const int64_t fwd[1][3] = {{s.D, s.Dv, G}}, bwd[3][3] = {{s.Dv, s.D, G}, {s.Dv, s.D, 1}, {s.D, s.Dv, 1}};
  plan_call(s, cus, 1, fwd, &p->fwd);
  plan_call(s, cus, 3, bwd, &p->bwd);
  const size_t states = (size_t)s.B * s.Hk * s.D * s.Dv * 4;
  p->total_fwd = p->step || p->fwd.segs == 1 ? 0 : align256_seq(states * p->fwd.segs);
  p->seg_bytes = p->bwd.segs == 1 ? 0 : align256_seq(states * p->bwd.segs);
  p->total_bwd = 3 * p->seg_bytes;
}

// The states at the segments' starts from the segments' own sums, in place:
// a thread an element, in the order of the run's time, eight segments' sums
// read ahead.
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
  const Decay decay = Decay::of(args.log_decay, hs);
  const int d = e / x.DV, c = e - d * x.DV;
  float S = x.s_in ? x.s_in[head * n + d * x.s_dk + c * x.s_dv] : 0.f;
  float* at = x.seg + head * args.segs * n + e;
  // decays of whole segments, of the one in which the sequence ends, of those past it
  const int whole = (int)(end / args.seg_rows);
  const Kept by_whole = decay.kept((int)args.seg_rows), by_rest = decay.kept((int)(end - whole * args.seg_rows)), all = {1.f, 0.f};
  constexpr int kAhead = 8;
  for (int o0 = 0; o0 < args.segs; o0 += kAhead) {
    float own[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) own[j] = o0 + j + 1 < args.segs ? at[(int64_t)(o0 + j) * n] : 0.f;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int o = o0 + j, seg = x.rev ? args.segs - 1 - o : o;
      if (o < args.segs) {
        at[(int64_t)o * n] = S;
        S = (seg < whole ? by_whole : seg == whole ? by_rest : all)(S, own[j]);
      }
    }
  }
}

static hipError_t launch_runs(int dtype, const LinArgs& a, const LinTile& t, int many, int dma, int64_t groups, hipStream_t s) {
  if (groups == 0) return hipSuccess;
  if (dtype == LSTM_F32) return launch_linattn_f32(a, t, many, dma, (unsigned)groups, s);
  if (dtype == LSTM_BF16) return launch_linattn_bf16(a, t, many, dma, (unsigned)groups, s);
  return launch_linattn_f16(a, t, many, dma, (unsigned)groups, s);
}

hipError_t launch_linattn(const LinPlan& p, const LinCall& c, LinArgs a, const int* dma, hipStream_t s) {
  a.segs = c.segs;
  a.seg_rows = c.seg_rows;
  // runs of one instance share a launch, those that share the state's update apart
  for (int pass = a.segs > 1 ? 0 : 1; pass < 2; ++pass) {
    auto alike = [&](int i, int j) {
      return c.tile[i].dp == c.tile[j].dp && c.tile[i].nw == c.tile[j].nw && c.tile[i].ks == c.tile[j].ks && dma[i] == dma[j] &&
             (pass == 0 || c.many[i] == c.many[j]);
    };
    bool done[3] = {false, false, false};
    for (int i = 0; i < a.runs; ++i) {
      if (done[i]) continue;
      LinArgs l = a;
      l.runs = 0;
      l.state_only = pass == 0;
      l.segs_of_launch = pass == 0 ? a.segs - 1 : a.segs;
      l.share = 0;
      for (int k = 0; k < 2 * a.runs; ++k) {  // those of summed heads first: they take longest
        const int j = k % a.runs;
        if (done[j] || !alike(i, j) || (a.run[j].gb > 1) != (k < a.runs)) continue;
        done[j] = true;
        LinRun& r = l.run[l.runs++];
        r = a.run[j];
        r.dv_blocks = (r.DV + 32 * c.tile[j].nw - 1) / (32 * c.tile[j].nw);
        r.member0 = l.share;
        l.share += r.dv_blocks * (pass == 0 || c.many[j] ? 1 : r.ga);
      }
      const int64_t groups = ((int64_t)a.B * a.Hs * l.segs_of_launch + 7) / 8 * 8 * l.share;
      const hipError_t e = launch_runs(p.dtype, l, c.tile[i], c.many[i], dma[i], groups, s);
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
// the bound.  A work-group has a (sequence, key head) and COLS columns of its
// state: COLS / 4 lanes of four columns each, the rows dealt to the other lanes.
constexpr int kStepHeads = 4;  // query heads at a time
template <typename T, int COLS, int RPT>
__global__ void __launch_bounds__(256) linattn_step_kernel(LinArgs args) {
  constexpr int CL = COLS / 4, RG = 256 / CL, HB = kStepHeads;
  constexpr int QN = HB * RPT * RG, QL = (QN + 255) / 256;  // values of q staged, and by a lane
  const LinRun& x = args.run[0];
  __shared__ float qs[HB][RPT * RG], ks[RPT * RG], vs[COLS];
  __shared__ f32x4_t part[HB][RG][CL];
  const int tid = threadIdx.x, cl = tid % CL, rg = tid / CL;
  const int dvb = (int)(blockIdx.x % (unsigned)x.dv_blocks);
  const int64_t head = blockIdx.x / (unsigned)x.dv_blocks;
  const int b = (int)(head / args.Hs), hs = (int)(head - (int64_t)b * args.Hs);
  const int dv0 = dvb * COLS, c0 = dv0 + 4 * cl;
  const bool whole = x.DV % 4 == 0 && ((uintptr_t)x.s_in & 15) == 0 && ((uintptr_t)x.s_out & 15) == 0;
  int end = (int)args.T;
  if (args.len) {
    const int l = args.len[b];
    end = l < 0 ? 0 : l < end ? l : end;
  }
  const Decay decay = Decay::of(args.log_decay, hs);

  // a step's k, v and first heads of q, read ahead (the first before the state:
  // loads return in order)
  float kx = 0.f, vx = 0.f, qx[QL];
  const int first_heads = x.ga < HB ? x.ga : HB;
  auto q_at = [&](int t, int g, int d) __attribute__((always_inline)) {
    return Elem<T>::load((const T*)x.a + t * x.as.t + b * x.as.b + (int64_t)(hs * x.ga + g) * x.as.h + d);
  };
  auto fetch = [&](int t) __attribute__((always_inline)) {
    if (t >= end) return;
    if (tid < x.DK) kx = Elem<T>::load((const T*)x.k + t * x.ks.t + b * x.ks.b + hs * x.ks.h + tid);
    if (tid < COLS && dv0 + tid < x.DV) vx = Elem<T>::load((const T*)x.v + t * x.vs.t + b * x.vs.b + hs * x.vs.h + dv0 + tid);
#pragma unroll
    for (int j = 0; j < QL; ++j) {
      const int g = (tid + 256 * j) / (RPT * RG), d = (tid + 256 * j) % (RPT * RG);
      if (g < first_heads && d < x.DK) qx[j] = q_at(t, g, d);
    }
  };
  fetch(0);

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
  const Kept kept = decay.kept(1);
  for (int t = 0; t < (int)args.T; ++t) {
    const bool real = t < end;
    if (real) {
      if (t > 0) __syncthreads();  // the step before has been read
      if (tid < x.DK) ks[tid] = kx;
      if (tid < COLS) vs[tid] = vx;
#pragma unroll
      for (int j = 0; j < QL; ++j)
        if (tid + 256 * j < QN) (&qs[0][0])[tid + 256 * j] = qx[j];
      fetch(t + 1);
    }
    for (int g0 = 0; g0 < x.ga; g0 += HB) {
      const int heads = x.ga - g0 < HB ? x.ga - g0 : HB;
      if (real) {
        if (g0 > 0) {
          __syncthreads();  // the heads before have been read
          for (int i = tid; i < heads * x.DK; i += 256) {
            const int g = i / x.DK, d = i - g * x.DK;
            qs[g][d] = q_at(t, g0 + g, d);
          }
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
              for (int j = 0; j < 4; ++j) S[r][j] = kept(S[r][j], k * v[j]);
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
      if (tid < heads * COLS) {  // (HB COLS threads at most)
        const int g = tid / COLS, c = tid % COLS;
        if (dv0 + c < x.DV) {
          float o = 0.f;
          if (real) {
#pragma unroll
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

// Small work-groups, whose reads and writes overlap other ones', but for heads
// that share a state or columns that are not divided, where a work-group's fixed
// work counts (32 and 64 columns, us from HBM: 256 sequences, 16 heads of 128 115
// and 132, 16 sequences 11.9 and 13.6; 256 sequences, 8/2 heads of 80 x 112 17.7 and
// 13.8; 200 sequences, 3 heads of 37 x 51 9.7 and 7.7).
template <typename T, int COLS>
static hipError_t step_launch(const LinArgs& a, unsigned groups, hipStream_t s) {
  constexpr int R = COLS / 32;  // rows of a lane per 32
  Timed timed(10, s);
  const int DK = a.run[0].DK;
  if (DK <= 64) linattn_step_kernel<T, COLS, 2 * R><<<dim3(groups), 256, 0, s>>>(a);
  else if (DK <= 96) linattn_step_kernel<T, COLS, 3 * R><<<dim3(groups), 256, 0, s>>>(a);
  else if (DK <= 128) linattn_step_kernel<T, COLS, 4 * R><<<dim3(groups), 256, 0, s>>>(a);
  else linattn_step_kernel<T, COLS, 8 * R><<<dim3(groups), 256, 0, s>>>(a);
  return hipGetLastError();
}
template <typename T>
static hipError_t step_of(const LinPlan& p, LinArgs a, hipStream_t s) {
  LinRun& x = a.run[0];
  const int64_t heads = (int64_t)a.B * a.Hs;
  const bool wide = (x.ga > 1 || x.DV <= 64) && heads * ((x.DV + 63) / 64) >= 2 * (int64_t)p.cus;
  const int cols = wide ? 64 : 32;
  x.dv_blocks = (x.DV + cols - 1) / cols;
  const int64_t groups = heads * x.dv_blocks;
  if (groups == 0) return hipSuccess;
  return wide ? step_launch<T, 64>(a, (unsigned)groups, s) : step_launch<T, 32>(a, (unsigned)groups, s);
}

hipError_t launch_linattn_step(const LinPlan& p, const LinArgs& a, hipStream_t s) {
  if (p.dtype == LSTM_F32) return step_of<float>(p, a, s);
  if (p.dtype == LSTM_BF16) return step_of<bf16_t>(p, a, s);
  return step_of<f16_t>(p, a, s);
}

}  // namespace lstm
