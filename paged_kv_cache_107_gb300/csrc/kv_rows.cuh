// kv_rows.cuh — the rows of new tokens on their way into a cache: rotary positions, 8-bit
// quantisation, the scatter by slot. store_q8.cu and rotary_store_*.cu instantiate it.
//
// A head's D dims are D/16 units of 16, one for each of the lanes that hold the head: a unit is
// two vectors of 8 elements, chosen so that both dims of a rotated pair lie in one lane (vectors
// u and u + R/16 for pairs R/2 apart, 2u and 2u + 1 for neighbours and for what passes
// through). A warp has one work item: up to kRowsUnroll groups of 32 / (D/16) heads of a token's
// queries, keys or values, all loaded before the first is used.
//
// Angles: position times the frequency's 64-bit fraction of a turn, modulo 2^64, is the angle
// without its whole turns; its top 32 bits go to sincospi in fp32. Far positions cost no
// accuracy. A lane computes two frequencies and the unit's eight come by shuffles.
//
// Quantisation: the row's largest magnitude from the 16-bit elements, two at a time (a NaN wins:
// its pattern, like infinity's, is above every finite number's).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dependent_launch.cuh"
#include "pa_device.cuh"
#include "pa_launch.h"
#include "q8.cuh"

namespace pa {
namespace {

constexpr int kRowsUnroll = 2;   // head groups of a work item
constexpr int kRowsThreads = 256;

// Eight 16-bit elements, by one 16-byte access or by elements. (Plain loads: q may be turned in
// place.)
__device__ __forceinline__ uint4 ld_vec8(const uint16_t* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void st_vec8(uint16_t* p, const uint4& v, bool vec) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[2 * i] = (uint16_t)(w[i] & 0xffffu);
    p[2 * i + 1] = (uint16_t)(w[i] >> 16);
  }
}

template <bool F16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (F16) {
    return f16x2_f2(w);
  } else {
    float2 f;
    bf16x2_to_f32(w, f.x, f.y);
    return f;
  }
}
template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  if constexpr (F16) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    return f32x2_to_bf16x2(lo, hi);
  }
}

// The unit's pairs (vectors a and b of 8 elements) turned by cos, sin of its eight frequencies.
template <bool F16, bool ADJ>
__device__ __forceinline__ void turn_unit(uint4& va, uint4& vb, const float (&c)[8],
                                          const float (&s)[8]) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&va);
  uint32_t* b = reinterpret_cast<uint32_t*>(&vb);
  if constexpr (ADJ) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? a[i & 3] : b[i & 3];
      const float2 x = widen2<F16>(w);
      w = narrow2<F16>(x.x * c[i] - x.y * s[i], x.y * c[i] + x.x * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = widen2<F16>(a[i]), y = widen2<F16>(b[i]);
      a[i] = narrow2<F16>(x.x * c[2 * i] - y.x * s[2 * i],
                          x.y * c[2 * i + 1] - y.y * s[2 * i + 1]);
      b[i] = narrow2<F16>(y.x * c[2 * i] + x.x * s[2 * i],
                          y.y * c[2 * i + 1] + x.y * s[2 * i + 1]);
    }
  }
}

// cos and sin of the token's angles: this lane's unit u holds frequencies 8u .. 8u + 7.
__device__ __forceinline__ void unit_angles(const RowsArgs& a, int64_t tok, int lane, int u,
                                            float (&c)[8], float (&s)[8]) {
  float cs[2], sn[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = 2 * lane + i;
    cs[i] = sn[i] = 0.f;
    if (f < a.rot.rotary_dim / 2) {
      int axis = __ldg(a.rot.axes + f);
      const uint64_t per_position = __ldg(a.rot.turns + f);
      if (axis < 0 || axis >= a.rot.num_axes) {
        set_dev_err(a.dev_err, PA_DEV_ERR_AXIS);
        axis = 0;
      }
      const int64_t p = __ldg(a.positions + axis * a.pos_stride + tok);
      const uint64_t turn = (uint64_t)p * per_position;
      float sv, cv;
      sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &sv, &cv);  // 2^-31
      cs[i] = cv * a.rot.amplitude;
      sn[i] = sv * a.rot.amplitude;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = __shfl_sync(0xffffffffu, cs[e & 1], 4 * u + (e >> 1));
    s[e] = __shfl_sync(0xffffffffu, sn[e & 1], 4 * u + (e >> 1));
  }
}

// The larger magnitudes of two pairs of elements; NaN wins.
template <bool F16>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (F16)
    asm("{\n\t.reg .b32 x, y;\n\tabs.f16x2 x, %1;\n\tabs.f16x2 y, %2;\n\tmax.NaN.f16x2 %0, x, y;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
  else
    asm("{\n\t.reg .b32 x, y;\n\tabs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.NaN.bf16x2 %0, x, y;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
  return r;
}

// FMT: 0 = 16-bit cache, else a pa_q8_format.
template <int D, bool F16, int FMT, bool ROT, bool ADJ>
__global__ void __launch_bounds__(kRowsThreads, ROT ? 5 : 8) kv_rows_kernel(const RowsArgs a) {
  constexpr int UNITS = D / 16;    // lanes of one head
  constexpr int HPW = 32 / UNITS;  // heads a warp moves at a time
  constexpr int U = kRowsUnroll;
  const int lane = threadIdx.x & 31;
  const int u = lane % UNITS;
  const int warp = threadIdx.x >> 5;
  // The warp's token and chunk of heads. 16-bit caches: a token's chunks follow each other. 8-bit
  // ones: a block takes one chunk of as many consecutive tokens as it has warps, whose scales it
  // writes together (without that need the first order is 4 % faster).
  constexpr bool kTogether = FMT != 0;
  const uint32_t chunks = (uint32_t)(a.q_chunks + 2 * a.kv_chunks);
  const uint32_t item = kTogether ? blockIdx.x : blockIdx.x * (blockDim.x / 32) + warp;
  const uint32_t group = item / chunks;
  int chunk = (int)(item - group * chunks);
  const int64_t my_tok = kTogether ? (int64_t)group * (blockDim.x / 32) + warp : (int64_t)group;

  pdl_launch_dependents();
  pdl_wait();
  const bool live = my_tok < a.num_tokens;
  if (!kTogether && !live) return;
  const int64_t tok = live ? my_tok : a.num_tokens - 1;
  const bool is_q = ROT && chunk < a.q_chunks;
  if (!is_q) chunk -= a.q_chunks;
  const bool is_v = !is_q && chunk >= a.kv_chunks;
  if (is_v) chunk -= a.kv_chunks;
  const int heads = is_q ? a.num_heads : a.num_kv_heads;
  const int h0 = chunk * (HPW * U) + lane / UNITS;

  // the vectors of this lane's unit: a pair's two dims lie in them
  const int half = a.rot.rotary_dim / 16;  // vectors, and units, that hold turned dims
  const bool turned = ROT && !is_v && u < half;
  const int va = 8 * ((!ADJ && turned) ? u : 2 * u);
  const int vb = 8 * ((!ADJ && turned) ? u + half : 2 * u + 1);
  const uint16_t* src = is_q ? static_cast<const uint16_t*>(a.q) + tok * a.q_stride
                        : is_v ? static_cast<const uint16_t*>(a.v) + tok * a.v_stride
                               : static_cast<const uint16_t*>(a.k) + tok * a.k_stride;
  const bool vec = a.vec != 0;
  const int64_t slot = live ? __ldg(a.slots + tok) : -1;
  uint4 xa[U], xb[U];
  auto load = [&](bool v) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      // (not under a condition of its own, which would put each load next to its use)
      const uint16_t* row = src + min(h0 + i * HPW, heads - 1) * D;
      xa[i] = ld_vec8(row + va, v);
      xb[i] = ld_vec8(row + vb, v);
    }
  };
  if (vec) load(true);
  else load(false);
  if constexpr (ROT) {
    if (!is_v) {
      float c[8], s[8];
      unit_angles(a, tok, lane, u, c, s);
      if (turned) {
#pragma unroll
        for (int i = 0; i < U; ++i) turn_unit<F16, ADJ>(xa[i], xb[i], c, s);
      }
    }
    if (is_q) {
      uint16_t* dst = static_cast<uint16_t*>(a.q_out) + tok * a.q_out_stride;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int h = h0 + i * HPW;
        if (h < heads && live) {
          st_vec8(dst + h * D + va, xa[i], vec);
          st_vec8(dst + h * D + vb, xb[i], vec);
        }
      }
      return;
    }
  }
  const bool keep = slot >= 0 && slot < a.num_slots;
  if (!keep && slot != -1 && lane == 0) set_dev_err(a.dev_err, PA_DEV_ERR_SLOT);
  if constexpr (FMT == 0) {
    uint16_t* dst = static_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) + slot * heads * D;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * HPW;
      if (h < heads && keep) {
        st_vec8(dst + h * D + va, xa[i], true);
        st_vec8(dst + h * D + vb, xb[i], true);
      }
    }
  } else {
    unsigned char* dst = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache) + slot * heads * D;
    // the block's scales, and its slots (-1: nothing is written)
    __shared__ float tok_scale[kRowsThreads / 32][HPW * U];
    __shared__ int32_t tok_slot[kRowsThreads / 32];
    if (lane == 0) tok_slot[warp] = keep ? (int32_t)slot : -1;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * HPW;
      const uint32_t* wa = reinterpret_cast<const uint32_t*>(&xa[i]);
      const uint32_t* wb = reinterpret_cast<const uint32_t*>(&xb[i]);
      uint32_t top = max_abs2<F16>(
          max_abs2<F16>(max_abs2<F16>(wa[0], wa[1]), max_abs2<F16>(wa[2], wa[3])),
          max_abs2<F16>(max_abs2<F16>(wb[0], wb[1]), max_abs2<F16>(wb[2], wb[3])));
#pragma unroll
      for (int m = 1; m < UNITS; m <<= 1)
        top = max_abs2<F16>(top, __shfl_xor_sync(0xffffffffu, top, m));
      top = max(top & 0xffffu, top >> 16);
      const RowScale r = row_scale<FMT>(widen2<F16>(top).x);
      const bool finite = r.scale == r.scale;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t* p = e < 2 ? wa + 2 * e : wb + 2 * (e - 2);
        const float2 lo = widen2<F16>(p[0]), hi = widen2<F16>(p[1]);
        w[e] = finite ? quantise4<FMT>(r, lo.x, lo.y, hi.x, hi.y) : 0u;
      }
      if (u == 0) tok_scale[warp][i * HPW + lane / UNITS] = r.scale;
      if (h < heads && keep) {
        if (vb == va + 8) {
          *reinterpret_cast<uint4*>(dst + h * D + va) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          *reinterpret_cast<uint2*>(dst + h * D + va) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(dst + h * D + vb) = make_uint2(w[2], w[3]);
        }
      }
    }
    // The scales of a head's consecutive tokens lie side by side where their slots do: written
    // together, 8 tokens fill a sector. (Four bytes at a time from every warp they cost 15 % of
    // the call: 66.8 us against 57.4 without them for 64,000 tokens of 8 heads of 128.)
    __syncthreads();
    const int lg_tokens = blockDim.x == kRowsThreads ? 3 : 1;  // warps of the block
    static_assert(kRowsThreads == 256, "eight warps, or two");
    if (threadIdx.x >= (HPW * U) << lg_tokens) return;
    const int t = threadIdx.x & ((1 << lg_tokens) - 1), hh = threadIdx.x >> lg_tokens;
    const int32_t s = tok_slot[t];
    const int h = chunk * (HPW * U) + hh;
    if (h < heads && s >= 0) {
      const uint32_t blk = (uint32_t)s / (uint32_t)a.block_size;
      (is_v ? a.v_scale : a.k_scale)[((int64_t)blk * heads + h) * a.block_size +
                                     ((uint32_t)s - blk * a.block_size)] = tok_scale[t][hh];
    }
  }
}

template <int D, bool F16, int FMT, bool ROT, bool ADJ>
int launch_rows_t(RowsArgs a, const DeviceInfo& info, cudaStream_t stream) {
  constexpr int per_item = 32 / (D / 16) * kRowsUnroll;
  a.q_chunks = ROT ? (int)(((int64_t)a.num_heads + per_item - 1) / per_item) : 0;
  a.kv_chunks = (int)(((int64_t)a.num_kv_heads + per_item - 1) / per_item);
  const int64_t chunks = a.q_chunks + 2 * (int64_t)a.kv_chunks;
  // few items are spread over the SMs in blocks of two warps
  const int threads = a.num_tokens * chunks < (int64_t)info.num_sms * 8 ? 64 : kRowsThreads;
  const int warps = threads / 32;
  const int64_t blocks = FMT == 0 ? (a.num_tokens * chunks + warps - 1) / warps
                                  : ((int64_t)a.num_tokens + warps - 1) / warps * chunks;
  // (a row of 2^31 elements is not memory that anyone has)
  if (a.num_tokens * chunks > INT32_MAX || blocks > INT32_MAX || ((int64_t)a.num_heads + per_item) * D > INT32_MAX ||
      ((int64_t)a.num_kv_heads + per_item) * D > INT32_MAX)
    return PA_ERR_UNSUPPORTED;
  if (launch_dependent(kv_rows_kernel<D, F16, FMT, ROT, ADJ>, dim3((unsigned)blocks),
                       dim3((unsigned)threads), 0, stream, a) != cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Every rotary form of one head_dim and element type.
template <int D, bool F16>
int launch_rotary_rows_t(const RowsArgs& a, int fmt, const DeviceInfo& info, cudaStream_t stream) {
  const bool adj = a.rot.adjacent != 0;
  switch (fmt) {
    case 0:
      return adj ? launch_rows_t<D, F16, 0, true, true>(a, info, stream)
                 : launch_rows_t<D, F16, 0, true, false>(a, info, stream);
    case PA_Q8_E4M3:
      return adj ? launch_rows_t<D, F16, PA_Q8_E4M3, true, true>(a, info, stream)
                 : launch_rows_t<D, F16, PA_Q8_E4M3, true, false>(a, info, stream);
    default:
      return adj ? launch_rows_t<D, F16, PA_Q8_INT8, true, true>(a, info, stream)
                 : launch_rows_t<D, F16, PA_Q8_INT8, true, false>(a, info, stream);
  }
}

}  // namespace
}  // namespace pa
