// shared_groups.cuh — the groups of pa_decode_shared on the device: which leading keys a
// group computes once, how that work is cut into steps, which CTAs of the one launch take it
// (prefix_body.cuh) and which the rest of the sequences (decode_tc.cuh).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

constexpr int kPrefixRows = 128;  // query rows per tile of the prefix part
constexpr int kPrefixKeys = 128;  // keys per tile

// Leading positions that a group of n sequences computes once: the prefix, where there are
// bytes to save. A lone sequence reads its keys once either way, and below a key tile there is
// nothing to multiply. The rule does not weigh time: a lone row tile of few rows costs its
// steps whatever n. 64 groups of n behind a prefix, together / each for itself (16 / 8 heads,
// head_dim 128): n = 2 42 / 27 us at 128 positions, 64 / 47 at 512, 78 / 89 at 1,024; n = 4
// 43 / 37, 64 / 96, 83 / 172; n = 16 73 / 103, 96 / 325, 133 / 637. (32 / 8 heads, head_dim 64:
// n = 2 36 / 21, 43 / 32, 63 / 48; n = 4 38 / 27, 49 / 51, 75 / 93.)
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
    if (i < n)  // (the prefix of an empty group is not looked at)
      bad = bad || starts[i] > starts[i + 1] ||
            (starts[i] < starts[i + 1] && (prefix[i] < 0 || prefix[i] > cap));
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
// tiles at a time (a step: two key tiles, one in each slot). A unit's start and end (its Q,
// the first products, the rows written out) cost about as much as kUnitSteps steps, which
// are counted before its own so that equal shares of the stream take equal times.
constexpr int kUnitSteps = 3;
struct GroupWork {
  int nt;      // key tiles
  int full;    // units per KV head with two row tiles
  int single;  // 1: one more with a single row tile

  __device__ __forceinline__ GroupWork(const SharedArgs& sh, int n, int prefix, int P) {
    const int len = shared_len(sh, n, prefix);
    nt = (len + kPrefixKeys - 1) / kPrefixKeys;
    const int tiles = (n + P - 1) / P;
    full = len > 0 ? tiles >> 1 : 0;
    single = len > 0 ? tiles & 1 : 0;
  }
  __device__ __forceinline__ int unit_steps(int pair) const {  // kUnitSteps included
    return kUnitSteps + (pair < full ? nt : (nt + 1) >> 1);
  }
  __device__ __forceinline__ int64_t steps(int Hk) const {
    return (int64_t)Hk * ((int64_t)full * (kUnitSteps + nt) +
                          (single ? kUnitSteps + ((nt + 1) >> 1) : 0));
  }
  // first step of unit (pair, KV head j), counted from the group's first
  __device__ __forceinline__ int64_t unit_first(int Hk, int pair, int j) const {
    return (int64_t)Hk * pair * (kUnitSteps + nt) + (int64_t)j * unit_steps(pair);
  }
};

// CTA c of g takes steps [c*nx/g, (c+1)*nx/g).
__device__ __forceinline__ int64_t prefix_begin(int64_t c, int64_t nx, int g) {
  return (c * nx) / g;
}
__device__ __forceinline__ int64_t prefix_cta_of(int64_t x, int64_t nx, int g) {
  return ((x + 1) * g - 1) / nx;
}

// The split of a launch, worked out by every CTA from the input arrays alone.
struct SharedPlan {
  bool ok;           // the arrays describe groups of the batch
  int64_t nx, nt;    // steps of the prefixes; key tiles of the rests
  int prefix_ctas;   // CTAs 0 .. prefix_ctas - 1 take the steps,
  int rest_ctas;     // the next rest_ctas of each KV head slab the tiles
  // in shared memory until the CTA's first copies
  const int *starts, *prefix;
  const int64_t* first_x;  // first step of each group
};

// Times on one SM in units of 0.1 us, from timelines of both parts: a step, bound by its
// products and softmax or by what one SM takes from memory (57 to 61 GB/s, measured with 8
// to 114 CTAs); a 64 KB tile of a rest; a rest's start and end. Side by side on the SMs instead
// of one after the other, the two parts share one start-up, and the steps' products run
// while the rests wait for memory: 50.7 -> 40 us for 64 sequences behind 8,192 keys, 117.5
// -> 113 us for 128 behind 32,768 (37 and 98 with the later steps).
constexpr int kStepCost = 18, kTileCost = 11, kRestCost = 20;
// A prefix CTA's start and end beyond a rest CTA's.
constexpr int kPrefixCtaCost = 33;
constexpr int kPrefixMinSteps = kUnitSteps + 2;

// Where one group makes up the prefixes and its units all have two row tiles: their number per
// KV head, else 1. The same share of every unit (a multiple of this many CTAs) lets the CTAs that
// read the same keys for other rows go through them side by side, so that all but one find them
// in L2 (128 sequences of 4 heads per KV head behind 32,768 keys: 528 -> 399 MB from memory, a
// step 1.71 -> 1.49 us, the launch 107 -> 98 us).
__device__ __forceinline__ int common_pairs(const SharedPlan& p, const SharedArgs& sh, int Hk,
                                            int P) {
  if (!p.ok || p.nx == 0) return 1;
  int lo = 0, hi = sh.num_groups - 1;  // the first group with steps: the last that starts at 0
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.first_x[mid] == 0) lo = mid;
    else hi = mid - 1;
  }
  const GroupWork w(sh, p.starts[lo + 1] - p.starts[lo], p.prefix[lo], P);
  return w.steps(Hk) == p.nx && w.single == 0 ? w.full : 1;
}

__device__ __forceinline__ void split_shared(SharedPlan& p, int ctas, int slabs, int min_tiles,
                                             int seqs, int pairs) {
  const int64_t want1 = (p.nx + kPrefixMinSteps - 1) / kPrefixMinSteps;
  const int64_t want2 = max((int64_t)1, (p.nt + min_tiles - 1) / min_tiles);
  int64_t g1 = 0;
  if (p.nx > 0) {
    // c1 / g1 + kPrefixCtaCost = c2 / (ctas - g1), in two rounds
    const float c1 = (float)p.nx * kStepCost;
    const float c2 = (float)(p.nt * kTileCost + (int64_t)seqs * kRestCost) * (float)slabs;
    float g = (float)ctas * (c1 / (c1 + c2));
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
      g = c1 / fmaxf((c1 + c2 + kPrefixCtaCost * g) / (float)ctas - kPrefixCtaCost,
                     c1 / (float)ctas);
    g1 = max((int64_t)1, min(min((int64_t)(g + 0.5f), want1), (int64_t)(ctas - slabs)));
  }
  const bool level = pairs > 1 && g1 >= 4 * pairs;
  if (level) g1 -= g1 % pairs;
  const int64_t g2 = max((int64_t)1, min(want2, (ctas - g1) / slabs));
  if (p.nx > 0) g1 = min(want1, ctas - g2 * slabs);  // what the rests leave
  if (level) g1 -= g1 % pairs;
  p.prefix_ctas = (int)g1;
  p.rest_ctas = (int)g2;
}

// Where the join finds every sequence's prefix parts; entries dealt to the launch's CTAs.
__device__ __forceinline__ void write_prefix_parts(const DecodeSharedArgs& a,
                                                   const SharedPlan& plan, int active_ctas,
                                                   int threads) {
  const int H = a.num_heads, Hk = a.num_kv_heads, G = H / Hk, P = kPrefixRows / G;
  for (int i = (int)(blockIdx.x + threadIdx.x * active_ctas); i < a.num_seqs * Hk;
       i += active_ctas * threads) {
    PrefixParts w{0, 0, 0, 0};
    if (plan.ok && plan.nx > 0) {
      const int b = i / Hk, j = i % Hk, g = group_of(plan.starts, a.sh.num_groups, b);
      const GroupWork work(a.sh, plan.starts[g + 1] - plan.starts[g], plan.prefix[g], P);
      if (work.nt > 0) {
        const int at = b - plan.starts[g], tile = at / P, pair = tile >> 1;
        const int64_t x = plan.first_x[g] + work.unit_first(Hk, pair, j);
        w.c0 = (int)prefix_cta_of(x + kUnitSteps, plan.nx, plan.prefix_ctas);
        w.n = (int)prefix_cta_of(x + work.unit_steps(pair) - 1, plan.nx, plan.prefix_ctas) -
              w.c0 + 1;
        w.row = (pair < work.full ? (tile & 1) * kPrefixRows : 0) + at % P * G;
      }
    }
    a.sh.prefix[i] = w;
  }
}

}  // namespace pa
