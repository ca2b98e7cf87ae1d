// shared_join.cu — the last launch of pa_decode_shared: every output row from its partial results.
//
// With normalised partial rows o_i and base-2 log-sum-exps l_i over disjoint sets of keys,
//   o = sum_i 2^(l_i - m) o_i / sum_i 2^(l_i - m),  m = max_i l_i.
// A row's parts are those of its group's prefix unit (one for each CTA that took steps of it) and
// the segments of its rest. They are summed in a fixed order in fp32: the result does not
// depend on which CTA finished first.
//
// One warp per (sequence, head), 4 or 2 dims per lane. Bound by latency: one round trip to L2
// brings where the parts lie and, read on the chance, the two whose place is known (the first
// of the prefix and of the rest); a second one up to 16 more, log-sum-exps and rows at once.
// The code runs once, cold: lane u works out where part u lies and the others get its offset
// by a shuffle, because 16 unrolled address calculations took 2.9 us to fetch.
// A kernel of its own because the parts of one row are many when few groups share a long
// prefix (152 CTAs over 8 KV heads leave 19), and joined inside the decode they held up the
// key stream of the warps that met them (54 us against 20 us of bytes for 64 sequences behind
// 8,192 keys).
#include "dependent_launch.cuh"
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

constexpr int kJoinWarps = 8;

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (F16) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    return f32x2_to_bf16x2(lo, hi);
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kJoinWarps * 32)
    shared_join_kernel(const DecodeSharedArgs a) {
  constexpr int E = D / 32;  // dims per lane
  constexpr int U = 16;      // parts loaded together
  const SharedArgs& sh = a.sh;
  const int H = a.num_heads, Hk = a.num_kv_heads, G = H / Hk;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);  // b * H + h
  const int b = row / H, h = row % H;
  // (a large grid's CTAs would still fill the SMs unevenly when the next call's arrive)
  if ((int)gridDim.x <= a.grid_ctas) pdl_launch_dependents();
  if (b >= a.num_seqs) return;
  pdl_wait();
  const RestSegments rest = sh.rest[b];
  const PrefixParts pre = sh.prefix[b * Hk + h / G];
  auto load = [&](const float* src, float* v) {
    src += lane * E;
    if constexpr (E == 4) {
      const float4 x = *reinterpret_cast<const float4*>(src);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(src);
      v[0] = x.x, v[1] = x.y;
    }
  };
  float acc[E], den, m;
  {
    float vp[E], vr[E];
    load(sh.first_o + (int64_t)row * D, vp);
    load(sh.rest_o + (int64_t)row * D, vr);
    float lp = sh.first_lse[row], lr = sh.rest_lse[row];
    // the row is written already (or, after a wait that ran out, never will be)
    if (rest.n < 0 || rest.c0 < 0 || rest.n > a.grid_ctas - rest.c0) return;
    if (pre.n == 0) lp = -INFINITY;
    if (rest.n == 0) lr = -INFINITY;
    m = fmaxf(lp, lr);
    const float wp = lp == -INFINITY ? 0.f : fast_exp2(lp - m);
    const float wr = lr == -INFINITY ? 0.f : fast_exp2(lr - m);
    den = wp + wr;
#pragma unroll
    for (int e = 0; e < E; ++e)
      acc[e] = (wp != 0.f ? wp * vp[e] : 0.f) + (wr != 0.f ? wr * vr[e] : 0.f);
  }
  // the parts that other CTAs carried on: the prefix's, then the rest's
  const int np = max(0, pre.n - 1), n = np + max(0, rest.n - 1);
  const int prow = pre.row + h % G;
  for (int i0 = 0; i0 < n; i0 += U) {
    const int i = min(i0 + (lane & (U - 1)), n - 1);
    const bool of_prefix = i < np;
    const int at = of_prefix ? (pre.c0 + 1 + i) * 256 + prow : (rest.c0 + 1 + i - np) * H + h;
    float l = (of_prefix ? sh.more_lse : a.part_lse)[at];
    if (i0 + lane >= n || lane >= U) l = -INFINITY;
    const float* mine = (of_prefix ? sh.more_o : a.part_o) + (int64_t)at * D;
    const int64_t off = mine - sh.more_o;
    float v[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) load(sh.more_o + __shfl_sync(0xffffffffu, off, u), v[u]);
    float bm = fmaxf(m, l);
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, s));
    const float scale = m == -INFINITY ? 0.f : fast_exp2(m - bm);
    den *= scale;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= scale;
    m = bm;
    const float wt = l == -INFINITY ? 0.f : fast_exp2(l - m);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = __shfl_sync(0xffffffffu, wt, u);  // 0 past the last part
      den += w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[u][e], acc[e]);
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  uint16_t* dst = static_cast<uint16_t*>(a.out) + (int64_t)row * D + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<F16>(acc[0] * inv, acc[1] * inv),
                                                pack2<F16>(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack2<F16>(acc[0] * inv, acc[1] * inv);
}

template <int D, bool F16>
int launch_join_t(const DecodeSharedArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.num_seqs * a.num_heads;
  const dim3 grid((unsigned)((rows + kJoinWarps - 1) / kJoinWarps));
  if (launch_dependent(shared_join_kernel<D, F16>, grid, dim3(kJoinWarps * 32), 0, stream, a) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

int launch_decode_shared(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  if (a.head_dim != 64 && a.head_dim != 128) return PA_ERR_UNSUPPORTED;
  const int rc = a.head_dim == 64 ? (a.f16 ? launch_shared_d64_f16(a, info, stream)
                                           : launch_shared_d64_bf16(a, info, stream))
                                  : (a.f16 ? launch_shared_d128_f16(a, info, stream)
                                           : launch_shared_d128_bf16(a, info, stream));
  if (rc != PA_OK) return rc;
  if (a.head_dim == 64) return a.f16 ? launch_join_t<64, true>(a, stream)
                                     : launch_join_t<64, false>(a, stream);
  return a.f16 ? launch_join_t<128, true>(a, stream) : launch_join_t<128, false>(a, stream);
}

}  // namespace pa
