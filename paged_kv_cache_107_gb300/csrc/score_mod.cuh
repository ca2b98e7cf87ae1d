// score_mod.cuh — the score rules of pa_decode_mod and pa_prefill_mod (ScoreModArgs): which
// keys a query sees, and the tanh of the cap.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

// The keys one query (or every query of a work unit) can see: [0, keep) and [low, hi), or
// simply [0, hi) without HIDDEN. Their tiles of T keys are numbered without the ones that
// lie wholly between keep and low, which are neither read nor multiplied.
template <bool HIDDEN>
struct KeySpan {
  int hi, low, keep;

  __device__ __forceinline__ int kept(int T) const {  // tiles that hold a key below keep
    return HIDDEN ? (min(keep, hi) + T - 1) / T : 0;
  }
  __device__ __forceinline__ int skipped(int T) const {  // hidden tiles between keep and low
    return HIDDEN ? max(0, min(low, hi) / T - kept(T)) : 0;
  }
  // Tiles to walk. (low < hi or keep >= hi holds for every rule: a query sees itself.)
  __device__ __forceinline__ int tiles(int T) const { return (hi + T - 1) / T - skipped(T); }
  __device__ __forceinline__ int first_key(int T, int tile) const {  // of a numbered tile
    return (tile < kept(T) ? tile : tile + skipped(T)) * T;
  }
  // some key of [k, k + n) lies below keep or at low or later
  __device__ __forceinline__ bool any_visible(int k, int n) const {
    return !HIDDEN || k < keep || k + n > low;
  }
};

__device__ __forceinline__ int mod_prefix(const ScoreModArgs& m, int s) {
  return m.prefix_lens ? max(0, __ldg(m.prefix_lens + s)) : 0;
}

// low and keep of a query of sequence s at position p (p < hi).
__device__ __forceinline__ void mod_span(KeySpan<true>& k, const ScoreModArgs& m, int s, int p) {
  if (m.window <= 0) return;
  k.low = max(0, p - m.window + 1);
  k.keep = max(m.sink, mod_prefix(m, s));
}

// tanh(u) for the score cap: kTanhPoly below |u| = 1; from there on 1 - 2 / (1 + e^(2u)) with
// the hardware's exp2 and reciprocal, about 2e-7 absolute. (The hardware's own tanh is off by
// 5e-4 relative, 0.02 in a score near a cap of 50.) NaN stays NaN, +-inf gives +-1.
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float cap_tanh(float u) {
  const float z = u * u;
  constexpr float c0 = kTanhPoly[0], c1 = kTanhPoly[1], c2 = kTanhPoly[2], c3 = kTanhPoly[3],
                  c4 = kTanhPoly[4], c5 = kTanhPoly[5];
  const float p = fmaf(fmaf(fmaf(fmaf(fmaf(c5, z, c4), z, c3), z, c2), z, c1), z, c0);
  const float far =
      fmaf(-2.f, fast_rcp(1.f + fast_exp2(u * (2.f * 1.4426950408889634f))), 1.f);
  return fabsf(u) < 1.f ? u * p : far;
}

}  // namespace pa
