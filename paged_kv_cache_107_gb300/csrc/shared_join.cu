// shared_join.cu — the last launch of pa_decode_shared: every output row from its partial results.
//
// With normalised partial rows o_i and base-2 log-sum-exps l_i over disjoint sets of keys,
//   o = sum_i 2^(l_i - m) o_i / sum_i 2^(l_i - m),  m = max_i l_i.
// A row's parts are those of its group's prefix unit (one for each CTA that took steps of it),
// then the segments of its rest. They are summed in that order in fp32: the result does
// not depend on which CTA finished first.
//
// One warp per (sequence, head), 4 or 2 dims per lane. Bound by latency: three dependent round
// trips to L2 (where the parts lie, their log-sum-exps, their rows). A kernel of its own
// because the parts of one row are many when few groups share a long prefix (152 CTAs over
// 8 KV heads leave 19), and joined inside the decode they held up the key stream of the
// warps that met them (54 us against 20 us of bytes for 64 sequences behind 8,192 keys).
#include "dependent_launch.cuh"
#include "pa_device.cuh"
#include "pa_launch.h"
#include "shared_groups.cuh"

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
  constexpr int U = 8;       // rows loaded together
  const SharedArgs& sh = a.sh;
  const int H = a.num_heads, Hk = a.num_kv_heads, G = H / Hk, P = kPrefixRows / G;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);  // b * H + h
  pdl_launch_dependents();
  if (row >= (int64_t)a.num_seqs * H) return;
  pdl_wait();
  const int b = (int)(row / H), h = (int)(row % H), kvh = h / G;
  const RestSegments rest = sh.rest[b];
  const PrefixWhere w = sh.where[b];
  // the row is written already (or, after a wait that ran out, never will be)
  if (rest.n < 0 || rest.c0 < 0 || rest.n > a.grid_ctas - rest.c0) return;
  const int64_t nx = *sh.steps;
  // prefix parts
  const GroupWork work(sh, w.n, w.prefix, P);
  int np = 0;
  int64_t pc0 = 0, prow = 0;
  if (work.nt > 0) {
    const int tile = (b - w.first) / P;
    const int64_t x = w.group_x + work.unit_first(Hk, tile >> 1, kvh);
    const int ctas = prefix_ctas(nx, sh.prefix_grid);
    pc0 = prefix_cta_of(x, nx, ctas);
    np = (int)(prefix_cta_of(x + work.unit_steps(tile >> 1) - 1, nx, ctas) - pc0) + 1;
    // (a row tile alone in its unit is stored as the first)
    prow = ((tile >> 1) < work.full ? (tile & 1) * kPrefixRows : 0) + ((b - w.first) % P) * G + h % G;
  }
  const int n = np + rest.n;
  // part i: its index among the rows stored by sequence or by CTA
  auto at = [&](int i, const float* first, const float* more, const float* rest0,
                const float* rest_more, int stride) -> const float* {
    if (i < np) return i == 0 ? first + row * stride : more + ((pc0 + i) * 256 + prow) * stride;
    i -= np;
    return i == 0 ? rest0 + row * stride : rest_more + ((int64_t)(rest.c0 + i) * H + h) * stride;
  };
  float m = -INFINITY, den = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float l = -INFINITY;
    if (i0 + lane < n)
      l = *at(i0 + lane, sh.first_lse, sh.more_lse, sh.rest_lse, a.part_lse, 1);
    float bm = fmaxf(m, l);
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, s));
    const float scale = m == -INFINITY ? 0.f : fast_exp2(m - bm);
    den *= scale;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= scale;
    m = bm;
    const float wt = l == -INFINITY ? 0.f : fast_exp2(l - m);
    const int nb = min(32, n - i0);
    for (int j0 = 0; j0 < nb; j0 += U) {
      float v[U][E], wj[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u;
        wj[u] = __shfl_sync(0xffffffffu, wt, j < nb ? j : 0);
        if (j >= nb) wj[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = 0.f;
        if (wj[u] != 0.f) {
          const float* src =
              at(i0 + j, sh.first_o, sh.more_o, sh.rest_o, a.part_o, D) + lane * E;
          if constexpr (E == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[u][0] = x.x, v[u][1] = x.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        den += wj[u];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wj[u], v[u][e], acc[e]);
      }
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  uint16_t* dst = static_cast<uint16_t*>(a.out) + row * D + lane * E;
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

int launch_shared_join(const DecodeSharedArgs& a, const DeviceInfo&, cudaStream_t stream) {
  if (a.head_dim == 64) return a.f16 ? launch_join_t<64, true>(a, stream)
                                     : launch_join_t<64, false>(a, stream);
  return a.f16 ? launch_join_t<128, true>(a, stream) : launch_join_t<128, false>(a, stream);
}

}  // namespace pa
