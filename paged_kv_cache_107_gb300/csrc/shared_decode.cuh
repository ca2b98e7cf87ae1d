// shared_decode.cuh — the launch of pa_decode_shared that reads the keys: the shared prefixes on
// the tcgen05 tensor cores (prefix_body.cuh) and the rest of every sequence on the warp
// tensor-core decode (decode_tc.cuh), side by side on the SMs. One CTA per SM; every CTA
// works out the same plan (SharedPlan) from the input arrays and takes its part.
#pragma once

#include "decode_tc.cuh"
#include "prefix_body.cuh"

namespace pa {
namespace {

constexpr int kPlanBytes = 4096;  // the scratch of the sums below; the plan's arrays follow

// Sums the work and splits the CTAs (all threads of the block).
template <int HS, int D>
__device__ __forceinline__ SharedPlan make_plan(const DecodeSharedArgs& a, unsigned char* smem) {
  constexpr int kWarps = kPrefillThreads / 32;
  constexpr int T = TcCfg<HS, D>::T;
  const SharedArgs& sh = a.sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = a.num_seqs, Hk = a.num_kv_heads, P = kPrefixRows / (a.num_heads / Hk);
  const int cap = a.max_blocks * a.block_size;
  int64_t* red_x = reinterpret_cast<int64_t*>(smem);
  int64_t* red_t = red_x + kWarps;
  int* starts = reinterpret_cast<int*>(smem + kPlanBytes);
  int* prefix = starts + sh.num_groups + 1;
  int64_t* first_x = reinterpret_cast<int64_t*>(starts + ((2 * sh.num_groups + 2) & ~1));
  const int ctx0 = tid < B ? __ldg(a.context_lens + tid) : 0;  // on its way beside the groups

  SharedPlan p;
  p.starts = starts;
  p.prefix = prefix;
  p.first_x = first_x;
  p.ok = load_groups(sh, B, cap, starts, prefix);
  if (!p.ok && blockIdx.x == 0 && tid == 0) set_dev_err(a.dev_err, PA_DEV_ERR_SEQLENS);
  // tiles of the rests
  int64_t nt = 0;
  for (int b = tid; b < B; b += kPrefillThreads) {
    const int raw = b == tid ? ctx0 : __ldg(a.context_lens + b);
    int low = 0;
    if (p.ok) {
      const int g = group_of(starts, sh.num_groups, b);
      low = shared_len(sh, starts[g + 1] - starts[g], prefix[g]);
    }
    // (or a context that ends inside its group's prefix)
    if ((raw < 0 || raw > cap || (raw > 0 && raw < low)) && b % (int)gridDim.x == (int)blockIdx.x)
      set_dev_err(a.dev_err, PA_DEV_ERR_CONTEXT);
    const int ctx = raw < 0 || raw > cap ? 0 : raw;
    if (ctx > low) nt += KeySpan<true>{ctx, low, 0}.tiles(T);
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) nt += __shfl_xor_sync(0xffffffffu, nt, m);
  if (lane == 0) red_t[warp] = nt;
  // steps of the prefixes: the first one of every group
  int64_t running = 0;
  for (int base = 0; base < sh.num_groups; base += kPrefillThreads) {
    const int g = base + tid;
    const int64_t n = p.ok && g < sh.num_groups
                          ? GroupWork(sh, starts[g + 1] - starts[g], prefix[g], P).steps(Hk)
                          : 0;
    int64_t incl = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += y;
    }
    if (base > 0) __syncthreads();
    if (lane == 31) red_x[warp] = incl;
    __syncthreads();
    int64_t before = running;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += red_x[w];
      running += red_x[w];
    }
    if (g < sh.num_groups) first_x[g] = before + incl - n;
  }
  p.nx = running;
  p.nt = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) p.nt += red_t[w];
  __syncthreads();
  split_shared(p, (int)gridDim.x, Hk / HS, a.min_tiles, B, common_pairs(p, sh, Hk, P));
  return p;
}

template <int HS, int D, bool F16>
__global__ void __launch_bounds__(kPrefillThreads, 1)
    shared_decode_kernel(const __grid_constant__ CUtensorMap tm_k1,
                         const __grid_constant__ CUtensorMap tm_v1,
                         const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const DecodeSharedArgs a,
                         const int box_rows, const int tb) {
  extern __shared__ __align__(1024) unsigned char shared_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kTmaWarp && lane < 5)
    umma::prefetch_tmap(lane == 0 ? &tm_k1 : lane == 1 ? &tm_v1 : lane == 2 ? &tm_q
                        : lane == 3 ? &tm_k : &tm_v);
  const SharedPlan plan = make_plan<HS, D>(a, shared_smem);
  const int slabs = a.num_kv_heads / HS, active = plan.prefix_ctas + plan.rest_ctas * slabs;
  // Where the call leaves SMs idle the join may be launched, and wait, there. Where it does not,
  // the join's CTAs would crowd on the SMs that finish first, and those of the next call would lie
  // on the SMs as they come free. But a CTA of a prefix and one of the rests on the two SMs of a
  // pair slow each other down (138 us instead of 98 for 128 sequences behind 32,768 keys with the
  // parts alternating), and a fresh launch puts consecutive CTAs on pairs: 106 -> 98 us back to
  // back, 62 -> 56 for 257 sequences in eight groups.
  // (The rests' CTAs signal early in any case; the launch waits for the prefixes' too.)
  if (active < (int)gridDim.x) pdl_launch_dependents();
  if ((int)blockIdx.x < plan.prefix_ctas) {
    prefix_body<D, F16>(tm_k1, tm_v1, tm_q, a, box_rows, shared_smem, plan, active);
    return;
  }
  const int r = (int)blockIdx.x - plan.prefix_ctas;
  if (r >= plan.rest_ctas * slabs || warp > kProducerWarp) return;  // 9 warps from here on
  decode_tc_body<HS, false, D, F16, kTcShared>(tm_k, tm_v, a, tb, shared_smem, r % plan.rest_ctas,
                                               r / plan.rest_ctas, plan.rest_ctas, &plan);
}

template <int HS, int D, bool F16>
int launch_shared_t(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  constexpr size_t kSmem = prefix_smem_bytes<D>() > TcCfg<HS, D>::SMEM ? prefix_smem_bytes<D>()
                                                                       : TcCfg<HS, D>::SMEM;
  static_assert(kSmem <= 232448, "shared memory budget (opt-in maximum)");
  static_assert(kPlanBytes + 16 * kMaxSharedSeqs + 16 <= TcCfg<HS, D>::STAGES * TcCfg<HS, D>::STAGE_BYTES,
                "the plan's arrays lie in the first stages");
  static std::atomic<bool> attr_done[64];  // zero-initialised: false
  if (info.device < 0 || info.device >= 64) return PA_ERR_CUDA;
  if ((size_t)info.max_smem_optin < kSmem) return PA_ERR_UNSUPPORTED;
  auto kernel = shared_decode_kernel<HS, D, F16>;
  if (!attr_done[info.device].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) !=
        cudaSuccess)
      return PA_ERR_CUDA;
    attr_done[info.device].store(true, std::memory_order_release);
  }
  const int G = a.num_heads / a.num_kv_heads;
  const int box = prefix_box_rows(a.block_size), tb = tc_box_tokens(a.block_size, TcCfg<HS, D>::T);
  CUtensorMap mk1, mv1, mq, mk, mv;
  auto slab_map = [&](CUtensorMap* m, const void* base, int tokens, int heads) {
    return make_slab_map(m, base, a.num_kv_heads, D, F16, a.block_size, a.num_blocks, tokens, heads);
  };
  // (block sizes without a box: the maps are made all the same, and not used)
  if (!slab_map(&mk1, a.k_cache, box ? box : 1, 1) || !slab_map(&mv1, a.v_cache, box ? box : 1, 1) ||
      !make_rows_map(&mq, a.q, a.num_seqs, a.num_heads, D, F16, G, kRows / G) ||
      !slab_map(&mk, a.k_cache, tb ? tb : 1, HS) || !slab_map(&mv, a.v_cache, tb ? tb : 1, HS))
    return PA_ERR_CUDA;
  if (launch_dependent(kernel, dim3((unsigned)a.grid_ctas), dim3(kPrefillThreads), kSmem, stream,
                       mk1, mv1, mq, mk, mv, a, box ? box : kKeys, tb) != cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Every head slab for one (D, element type) combination.
template <int D, bool F16>
int dispatch_shared(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  switch (decode_head_slab(a.num_kv_heads)) {
    case 8: return launch_shared_t<8, D, F16>(a, info, stream);
    case 4: return launch_shared_t<4, D, F16>(a, info, stream);
    case 2: return launch_shared_t<2, D, F16>(a, info, stream);
    default: return launch_shared_t<1, D, F16>(a, info, stream);
  }
}

}  // namespace
}  // namespace pa
