// linattn_decay.hpp -- powers of a head's decay (gfx950).
#pragma once
#include "seq_internal.hpp"

namespace lstm {

// What a state keeps over some steps and what comes to it: a^n S + x, with a^n
// near 1 taken as 1 and the rest, whose rounding is relative to the rest.  A
// decay is applied to a state thousands of times, and the error of a fp32 a^n,
// up to 2^-25, would add up (4096 single tokens of memories of 3000 to 60000
// steps: 5.8e-5 of the state, so 8e-7).
struct Kept {
  float one, rest;  // 1 or 0, and a^n less it
  __device__ __forceinline__ float operator()(float S, float x) const {
    return __builtin_fmaf(S, one, __builtin_fmaf(S, rest, x));
  }
};

// a = exp(min(log_decay, 0)) of a head
struct Decay {
  float ln, log2;
  __device__ __forceinline__ static Decay of(const float* log_decay, int head) {
    const float x = log_decay[head], ln = x > 0.f ? 0.f : x;
    return {ln, ln * kLog2e};
  }
  // a^e of a whole e >= 0 (log2 is -inf for a decay of 0)
  __device__ __forceinline__ float power(int e) const { return e == 0 ? 1.f : __builtin_amdgcn_exp2f(log2 * (float)e); }
  // a^e - 1 where it is near 0, by its series: |x| <= 1/16, the next term is 2^-29
  // of the sum (else the state is gone after some hundred times)
  __device__ __forceinline__ static bool near(float x) { return x >= -0.0625f; }
  __device__ __forceinline__ static float less_one(float x) {
    return x * (1.f + x * (1.f / 2 + x * (1.f / 6 + x * (1.f / 24 + x * (1.f / 120)))));
  }
  __device__ __forceinline__ Kept kept(int e) const {
    const float x = e == 0 ? 0.f : ln * (float)e;
    return near(x) ? Kept{1.f, less_one(x)} : Kept{0.f, power(e)};
  }
  // a^e less `rounded`, the fp32 number that stands for it
  __device__ __forceinline__ float beyond(int e, float rounded) const {
    const float x = ln * (float)e;
    return near(x) ? less_one(x) - (rounded - 1.f) : 0.f;
  }
};

}  // namespace lstm
