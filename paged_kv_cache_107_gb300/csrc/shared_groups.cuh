// shared_groups.cuh — the groups of pa_decode_shared on the device: which leading keys a
// group computes once, how the prefix kernel cuts that work into steps, and where its
// partial results lie. Shared by the prefix kernel (prefix_kernel.cuh) and the decode of the
// rest (decode_tc.cuh), which both derive everything from the same two input arrays.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

constexpr int kPrefixRows = 128;  // query rows per tile of the prefix kernel
constexpr int kPrefixKeys = 128;  // keys per tile

// Leading positions that a group of n sequences computes once: the prefix, where there is
// something to save. A lone sequence reads its keys once either way.
__device__ __forceinline__ int shared_len(const SharedArgs& sh, int n, int prefix) {
  return sh.boxes && n >= 2 && prefix >= kPrefixKeys ? prefix : 0;
}

// Copies group_starts and prefix_lens to shared memory (starts[num_groups + 1], then
// prefix[num_groups]) and checks them; the whole block calls it. false: the arrays do not
// describe groups of the batch, and nothing is shared (the call still decodes every
// sequence, and the caller records the error).
__device__ __forceinline__ bool load_groups(const SharedArgs& sh, int B, int cap, int* starts,
                                            int* prefix) {
  const int n = sh.num_groups;
  for (int i = threadIdx.x; i <= n; i += blockDim.x) {
    starts[i] = __ldg(sh.group_starts + i);
    if (i < n) prefix[i] = __ldg(sh.prefix_lens + i);
  }
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i <= n; i += blockDim.x) {
    if (i < n) bad = bad || starts[i] > starts[i + 1] || prefix[i] < 0 || prefix[i] > cap;
    if (i == 0) bad = bad || starts[0] != 0;
    if (i == n) bad = bad || starts[n] != B;
  }
  return __syncthreads_or(bad) == 0;
}

// Group of sequence b: the last one that starts at b or before (the empty ones before it
// start at b too).
__device__ __forceinline__ int group_of(const int* starts, int num_groups, int b) {
  int lo = 0, hi = num_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (starts[mid] <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The prefix work of one group. Its query rows (sequences x the G heads of a KV head) fill
// tiles of P sequences; a unit is one KV head with two tiles that take every key tile
// together (a step: one key tile for both), or the last tile alone, which takes two key
// tiles at a time (a step: two key tiles, one in each slot of the kernel).
struct GroupWork {
  int nt;     // key tiles
  int full;   // units per KV head with two row tiles
  int single; // 1: one more with a single row tile

  __device__ __forceinline__ GroupWork(const SharedArgs& sh, int n, int prefix, int P) {
    const int len = shared_len(sh, n, prefix);
    nt = (len + kPrefixKeys - 1) / kPrefixKeys;
    const int tiles = (n + P - 1) / P;
    full = len > 0 ? tiles >> 1 : 0;
    single = len > 0 ? tiles & 1 : 0;
  }
  __device__ __forceinline__ int unit_steps(int pair) const {
    return pair < full ? nt : (nt + 1) >> 1;
  }
  __device__ __forceinline__ int64_t steps(int Hk) const {
    return (int64_t)Hk * ((int64_t)full * nt + (single ? (nt + 1) >> 1 : 0));
  }
  // first step of unit (pair, KV head j), counted from the group's first
  __device__ __forceinline__ int64_t unit_first(int Hk, int pair, int j) const {
    return (int64_t)Hk * pair * nt + (int64_t)j * unit_steps(pair);
  }
};

// CTAs that take steps of a stream of nx: at least kPrefixMinSteps each.
constexpr int kPrefixMinSteps = 2;
__device__ __forceinline__ int prefix_ctas(int64_t nx, int grid) {
  const int64_t want = (nx + kPrefixMinSteps - 1) / kPrefixMinSteps;
  return (int)(want < (int64_t)grid ? want : (int64_t)grid);
}
// CTA c of g takes steps [c*nx/g, (c+1)*nx/g).
__device__ __forceinline__ int64_t prefix_begin(int64_t c, int64_t nx, int g) {
  return (c * nx) / g;
}
__device__ __forceinline__ int64_t prefix_cta_of(int64_t x, int64_t nx, int g) {
  return ((x + 1) * g - 1) / nx;
}

}  // namespace pa
