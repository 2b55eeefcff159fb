// model_internal.hpp -- plans and launchers of linear attention, the logits'
// penalties and the AdamW step, which model_api.hip calls.
#pragma once
#include "seq_internal.hpp"

namespace lstm {

// ---- linattn.hip, linattn_common.hpp ----
// One recurrence over a call's sequences (linattn_common.hpp): rows a and keys
// k of DK values, values v and outputs of DV.
struct LinRun {
  const void *a, *k, *v;
  void* out;
  lstm_stride as, ks, vs, os;
  int DK, DV;
  int ga, gb;       // heads of a, of k and v, that share a state (one of them 1)
  int rev;          // backwards in time
  const float* s_in;  // [B][Hs] states before the first step, element (dk, dv) at dk s_dk + dv s_dv; null: zeros
  float* s_out;       // after the last, or null
  int64_t s_dk, s_dv;
  float* seg;       // [B][Hs][segs][DK][DV] states at the segments' starts
  int whole;        // kWholeQ / K / V / O of a, k, v, out
  int dv_blocks;    // work-groups a head's columns are split over
  uint32_t member0;  // first of its work-groups among a state's
};
struct LinArgs {
  LinRun run[3];
  int runs;
  uint32_t share;  // work-groups of the launch for a state (and segment), of all runs
  int64_t T;
  int B, Hs;
  const float* log_decay;  // [Hs]
  const int32_t* len;      // [B] or null
  float scale;
  int segs, segs_of_launch;  // segments of the time axis; those of this launch, from the run's first
  int64_t seg_rows;          // steps of a segment, a multiple of 32
  int state_only;            // the segments' own sums into seg, no outputs
};
// An instance of the kernel: the row size it runs with, 32-column tiles and parts
// of the state's rows of a work-group, a wave each.
struct LinTile {
  int dp, nw, ks;
};
struct LinCall {        // the forward, or the backward
  LinTile tile[3];     // of each run
  int many[3];
  int segs;            // segments of the time axis
  int64_t seg_rows;
};
struct LinPlan {
  int dtype, cus;
  LinCall fwd, bwd;
  int step;            // forward by the kernel for a few steps
  size_t seg_bytes;    // of one run's seg of the backward
  size_t total_fwd, total_bwd;
};
void make_linattn_plan(const lstm_linattn_shape& s, int cus, LinPlan* p);
// runs of a call, their seg set; dma[i]: rows of run i are whole aligned chunks
hipError_t launch_linattn(const LinPlan& p, const LinCall& c, LinArgs a, const int* dma, hipStream_t s);
hipError_t launch_linattn_step(const LinPlan& p, const LinArgs& a, hipStream_t s);
hipError_t launch_linattn_f32(const LinArgs& a, const LinTile& t, int many, int dma, unsigned groups, hipStream_t s);
hipError_t launch_linattn_bf16(const LinArgs& a, const LinTile& t, int many, int dma, unsigned groups, hipStream_t s);
hipError_t launch_linattn_f16(const LinArgs& a, const LinTile& t, int many, int dma, unsigned groups, hipStream_t s);

// ---- penalty.hip ----
struct PenaltyArgs {
  const void* logits;
  const void* history;
  const int32_t* length;
  const float *repetition, *presence, *frequency, *bias;
  const uint32_t* mask;
  void* out;
  int64_t N, V, ld, ldo, L, hn, ht, ldb, ldm;
  int dtype, id64;
  int64_t slice;  // logits of a work-group
  int slices;     // work-groups of a row
};
void make_penalty_plan(int cus, PenaltyArgs* a);
hipError_t launch_penalty(const PenaltyArgs& a, hipStream_t s);

// ---- adamw.hip ----
constexpr int kAdamwBlock = 256;   // values of an 8-bit state that share a scale
constexpr int kAdamwTensors = 48;  // tensors of a launch: their table is the kernel's argument (below 4 KB)
struct AdamwPlan {
  double lr, b1, b2, eps;
  int64_t step;
  int dtype, bits;
};
// values of a work-group of the norm's first launch, whose sums the second adds up
constexpr int64_t kNormChunk = 16384;
hipError_t launch_adamw_step(const AdamwPlan& p, const lstm_adamw_tensor* t, int64_t count,
                             const lstm_adamw_control* control, hipStream_t s);
hipError_t launch_adamw_norm(const AdamwPlan& p, const lstm_adamw_tensor* t, int64_t count, double max_norm,
                             double unscale, double* ws, lstm_adamw_control* control, hipStream_t s);

}  // namespace lstm
