// kv_rows.cuh — the rows of new tokens on their way into a cache: rotary positions, 8-bit
// quantisation, the scatter by slot. store_q8.cu and rotary_store_*.cu instantiate it.
//
// A head's D dims are D/16 units of 16, one for each of the lanes that hold the head: a unit is
// two vectors of 8 elements, chosen so that both dims of a rotated pair lie in one lane (vectors
// u and u + R/16 for pairs R/2 apart, 2u and 2u + 1 for neighbours and for what passes
// through). A warp has one work item: kRowsUnroll groups of 32 / (D/16) heads, of a token's
// queries, keys or values, or of consecutive rows of several tokens, all loaded before the first
// is used.
//
// Angles: position times the frequency's 64-bit fraction of a turn, modulo 2^64, is the angle
// without its whole turns; its top 32 bits go to sincospi in fp32. Far positions cost no
// accuracy. A lane computes two frequencies and the unit's eight come by shuffles.
//
// Quantisation: the row's largest magnitude from the 16-bit elements, two at a time (a NaN wins:
// its pattern, like infinity's, is above every finite number's).
//
// Bound by bytes: 17,556 tokens of 16 / 8 heads of 128 are turned and stored in 43.4 us, 6.6 TB/s
// or 0.98 of the copy rate; their keys and values quantised in 17.7 us (e4m3) and 18.5 (int8,
// whose instructions take 80 % of the issue slots), 64,000 tokens in 57 and 59 (1.02, 0.99). Turned
// and quantised in one launch the first take 43.8 us (e4m3) and 45.6 (int8; 73 % of the issue slots)
// of which the bytes are 37.3; in two, 60.7 and 61.3. Each
// warp has one item and the grid as many blocks as that takes: one resident wave of blocks that
// stride over the tokens was slower (49.8 us, 24.3), and so were items of 4 (46.8, 31.3) or of one
// (50.2, 24.0) groups.
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

// cos and sin, times the amplitude, of a frequency's angle at a position.
__device__ __forceinline__ void turn_angle(int32_t position, uint64_t per_position,
                                           float amplitude, float* c, float* s) {
  const uint64_t turn = (uint64_t)(int64_t)position * per_position;
  float sv, cv;
  sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &sv, &cv);  // 2^-31
  *c = cv * amplitude;
  *s = sv * amplitude;
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
      turn_angle(__ldg(a.positions + axis * a.pos_stride + tok), per_position, a.rot.amplitude,
                 &cs[i], &sn[i]);
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

template <int D>
struct RowsCfg {
  static constexpr int UNITS = D / 16;           // lanes of one head
  static constexpr int HPW = 32 / UNITS;         // heads a warp moves at a time
  static constexpr int R = HPW * kRowsUnroll;    // heads of a work item
  static constexpr int WARPS = kRowsThreads / 32;
};

// The two vectors of a lane's unit, by offset in a row, and whether they hold turned dims.
struct UnitPlace {
  int va, vb;
  bool turned;
};
template <bool ROT, bool ADJ>
__device__ __forceinline__ UnitPlace unit_place(const RowsArgs& a, int u, bool is_v) {
  const int half = a.rot.rotary_dim / 16;  // vectors, and units, that hold turned dims
  UnitPlace p;
  p.turned = ROT && !is_v && u < half;
  p.va = 8 * ((!ADJ && p.turned) ? u : 2 * u);
  p.vb = 8 * ((!ADJ && p.turned) ? u + half : 2 * u + 1);
  return p;
}

// Quantises the row whose units xa, xb its lanes hold; writes this lane's codes where `write`.
// Returns the row's scale.
template <int D, bool F16, int FMT>
__device__ __forceinline__ float quantise_unit(const uint4& xa, const uint4& xb,
                                               const UnitPlace& p, unsigned char* row, bool write) {
  const uint32_t* wa = reinterpret_cast<const uint32_t*>(&xa);
  const uint32_t* wb = reinterpret_cast<const uint32_t*>(&xb);
  uint32_t top =
      max_abs2<F16>(max_abs2<F16>(max_abs2<F16>(wa[0], wa[1]), max_abs2<F16>(wa[2], wa[3])),
                    max_abs2<F16>(max_abs2<F16>(wb[0], wb[1]), max_abs2<F16>(wb[2], wb[3])));
#pragma unroll
  for (int m = 1; m < RowsCfg<D>::UNITS; m <<= 1)
    top = max_abs2<F16>(top, __shfl_xor_sync(0xffffffffu, top, m));
  top = max(top & 0xffffu, top >> 16);
  const RowScale r = row_scale<FMT>(widen2<F16>(top).x);
  const bool finite = r.scale == r.scale;
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t* q = e < 2 ? wa + 2 * e : wb + 2 * (e - 2);
    const float2 lo = widen2<F16>(q[0]), hi = widen2<F16>(q[1]);
    w[e] = finite ? quantise4<FMT>(r, lo.x, lo.y, hi.x, hi.y) : 0u;
  }
  if (write) {
    if (p.vb == p.va + 8) {
      *reinterpret_cast<uint4*>(row + p.va) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(row + p.va) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + p.vb) = make_uint2(w[2], w[3]);
    }
  }
  return r.scale;
}

__device__ __forceinline__ void write_scale(float* scales, int32_t slot, int64_t heads, int h,
                                            int block_size, float scale) {
  const uint32_t blk = (uint32_t)slot / (uint32_t)block_size;
  scales[(blk * heads + h) * block_size + ((uint32_t)slot - blk * block_size)] = scale;
}

// Work items of one token each: every lane of the warp needs the same token's angles.
template <int D, bool F16, int FMT, bool ROT, bool ADJ>
__device__ __forceinline__ void wide_rows(const RowsArgs& a) {
  using C = RowsCfg<D>;
  constexpr int U = kRowsUnroll;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane % C::UNITS;
  // The warp's token and chunk of heads. 16-bit caches: a token's chunks follow each other. 8-bit
  // ones: a block takes one chunk of as many consecutive tokens as it has warps, whose scales it
  // writes together (without that need the first order is 4 % faster).
  constexpr bool kTogether = FMT != 0;
  const uint32_t chunks = (uint32_t)(a.q_chunks + 2 * a.kv_chunks);
  const uint32_t item = kTogether ? blockIdx.x : blockIdx.x * (blockDim.x / 32) + warp;
  const uint32_t group = item / chunks;
  int chunk = (int)(item - group * chunks);
  const int64_t my_tok = kTogether ? (int64_t)group * (blockDim.x / 32) + warp : (int64_t)group;
  const bool live = my_tok < a.num_tokens;
  if (!kTogether && !live) return;
  const int64_t tok = live ? my_tok : a.num_tokens - 1;
  const bool is_q = ROT && chunk < a.q_chunks;
  if (!is_q) chunk -= a.q_chunks;
  const bool is_v = !is_q && chunk >= a.kv_chunks;
  if (is_v) chunk -= a.kv_chunks;
  const int heads = is_q ? a.num_heads : a.num_kv_heads;
  const int h0 = chunk * C::R + lane / C::UNITS;
  const UnitPlace p = unit_place<ROT, ADJ>(a, u, is_v);
  const uint16_t* src = (is_q ? static_cast<const uint16_t*>(a.q) + tok * a.q_stride
                         : is_v ? static_cast<const uint16_t*>(a.v) + tok * a.v_stride
                                : static_cast<const uint16_t*>(a.k) + tok * a.k_stride);
  const bool vec = a.vec != 0;
  const int64_t slot = live ? __ldg(a.slots + tok) : -1;
  // (rotary calls: a second group without a head is not loaded, 11.0 -> 10.7 us for 4,095 tokens of
  // 32 / 8 heads of 64; alone, the quantising store is slower for the branch)
  const bool two = !ROT || chunk * C::R + C::HPW < heads;
  uint4 xa[U], xb[U];
  auto load = [&](bool v, int n) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      // (not under a condition of its own, which would put each load next to its use)
      const uint16_t* row = src + min(h0 + i * C::HPW, heads - 1) * D;
      xa[i] = ld_vec8(row + p.va, v);
      xb[i] = ld_vec8(row + p.vb, v);
    }
  };
  if (ROT) xa[1] = xb[1] = make_uint4(0u, 0u, 0u, 0u);
  if (vec && two) load(true, U);
  else if (vec) load(true, 1);
  else load(false, U);
  if constexpr (ROT) {
    if (!is_v) {
      float c[8], s[8];
      unit_angles(a, tok, lane, u, c, s);
      if (p.turned) {
#pragma unroll
        for (int i = 0; i < U; ++i) turn_unit<F16, ADJ>(xa[i], xb[i], c, s);
      }
    }
    if (is_q) {
      uint16_t* dst = static_cast<uint16_t*>(a.q_out) + tok * a.q_out_stride;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int h = h0 + i * C::HPW;
        if (h < heads && live) {
          st_vec8(dst + h * D + p.va, xa[i], vec);
          st_vec8(dst + h * D + p.vb, xb[i], vec);
        }
      }
      return;
    }
  }
  const bool keep = slot >= 0 && slot < a.num_slots;
  if (!keep && slot != -1 && lane == 0) set_dev_err(a.dev_err, PA_DEV_ERR_SLOT);
  const int64_t at = slot * heads * D;
  if constexpr (FMT == 0) {
    uint16_t* dst = static_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) + at;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * C::HPW;
      if (h < heads && keep) {
        st_vec8(dst + h * D + p.va, xa[i], true);
        st_vec8(dst + h * D + p.vb, xb[i], true);
      }
    }
  } else {
    unsigned char* dst = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache) + at;
    // The scales of a head's consecutive tokens lie side by side where their slots do: written
    // together, 8 tokens fill a sector. (Four bytes at a time from every warp they cost 15 % of
    // the call: 66.8 us against 57.4 without them for 64,000 tokens of 8 heads of 128.)
    // The block's scales, and its slots (-1: nothing is written):
    __shared__ float tok_scale[C::WARPS][C::R];
    __shared__ int32_t tok_slot[C::WARPS];
    if (lane == 0) tok_slot[warp] = keep ? (int32_t)slot : -1;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * C::HPW;
      const float scale =
          quantise_unit<D, F16, FMT>(xa[i], xb[i], p, dst + h * D, h < heads && keep);
      if (u == 0) tok_scale[warp][i * C::HPW + lane / C::UNITS] = scale;
    }
    __syncthreads();
    const int lg_tokens = blockDim.x == kRowsThreads ? 3 : 1;  // warps of the block
    static_assert(C::WARPS == 8, "eight warps, or two");
    if (threadIdx.x >= C::R << lg_tokens) return;
    const int t = threadIdx.x & ((1 << lg_tokens) - 1), hh = threadIdx.x >> lg_tokens;
    if (tok_slot[t] >= 0 && chunk * C::R + hh < heads)
      write_scale(is_v ? a.v_scale : a.k_scale, tok_slot[t], heads, chunk * C::R + hh,
                  a.block_size, tok_scale[t][hh]);
  }
}

// Blocks of consecutive rows (token, head) of the queries, the keys or the values, whatever the
// head count: a warp's rows may be of several tokens. The angles of the block's tokens are worked
// out once, in shared memory. For head counts that would leave too many lanes of wide items without
// a row (launch_rows_t has the rule): 32,000 tokens of 1 / 1 heads of 128 take 17.3 us, in wide items
// 35.4; quantised alone 6.6 and 27.5.
template <int D, bool F16, int FMT, bool ROT, bool ADJ>
__device__ __forceinline__ void flat_rows(const RowsArgs& a, uint32_t blk, bool is_q, bool is_v) {
  using C = RowsCfg<D>;
  constexpr int U = kRowsUnroll;
  constexpr int F = D / 2;  // most frequencies
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane % C::UNITS;
  const uint32_t heads = (uint32_t)(is_q ? a.num_heads : a.num_kv_heads);
  const uint64_t per_head = is_q ? a.q_magic : a.kv_magic;
  const uint32_t total = (uint32_t)a.num_tokens * heads;  // below 2^31 (the launcher)
  const uint32_t rows = C::R * (blockDim.x / 32);
  const uint32_t row0 = blk * rows;
  auto token_of = [&](uint32_t r) {
    return per_head ? (uint32_t)__umul64hi((uint64_t)r, per_head) : r;
  };
  const uint32_t tok0 = token_of(row0);
  const UnitPlace p = unit_place<ROT, ADJ>(a, u, is_v);
  const uint16_t* src = static_cast<const uint16_t*>(is_q ? a.q : is_v ? a.v : a.k);
  const int64_t stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
  const bool vec = a.vec != 0;
  const uint32_t r0 = row0 + warp * C::R + lane / C::UNITS;  // this lane's rows: + i HPW
  uint32_t tok[U], head[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t r = min(r0 + i * C::HPW, total - 1);
    tok[i] = token_of(r);
    head[i] = r - tok[i] * heads;
  }
  uint4 xa[U], xb[U];
  auto load = [&](bool v) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint16_t* row = src + tok[i] * stride + head[i] * D;
      xa[i] = ld_vec8(row + p.va, v);
      xb[i] = ld_vec8(row + p.vb, v);
    }
  };
  if (vec) load(true);
  else load(false);
  int64_t slot[U];
  if (!is_q) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      slot[i] = r0 + i * C::HPW < total ? __ldg(a.slots + tok[i]) : -1;
  }
  const uint32_t tokens = token_of(min(row0 + rows, total) - 1) - tok0 + 1;  // of the block
  if constexpr (ROT) {
    if (!is_v) {
      // at most as many tokens as rows
      __shared__ __align__(16) float cs[C::R * C::WARPS][F], sn[C::R * C::WARPS][F];
      const int f = threadIdx.x % F;
      if (f < a.rot.rotary_dim / 2) {
        int axis = __ldg(a.rot.axes + f);
        const uint64_t per_position = __ldg(a.rot.turns + f);
        if (axis < 0 || axis >= a.rot.num_axes) {
          set_dev_err(a.dev_err, PA_DEV_ERR_AXIS);
          axis = 0;
        }
        const int32_t* pos = a.positions + axis * a.pos_stride + tok0;
        for (uint32_t t = threadIdx.x / F; t < tokens; t += blockDim.x / F)
          turn_angle(__ldg(pos + t), per_position, a.rot.amplitude, &cs[t][f], &sn[t][f]);
      }
      __syncthreads();
      if (p.turned) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float4* cp = reinterpret_cast<const float4*>(&cs[tok[i] - tok0][8 * u]);
          const float4* sp = reinterpret_cast<const float4*>(&sn[tok[i] - tok0][8 * u]);
          const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
          const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
          turn_unit<F16, ADJ>(xa[i], xb[i], c, s);
        }
      }
    }
    if (is_q) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (r0 + i * C::HPW < total) {
          uint16_t* row =
              static_cast<uint16_t*>(a.q_out) + tok[i] * a.q_out_stride + head[i] * D;
          st_vec8(row + p.va, xa[i], vec);
          st_vec8(row + p.vb, xb[i], vec);
        }
      }
      return;
    }
  }
  void* cache = is_v ? a.v_cache : a.k_cache;
  __shared__ float row_scales[FMT != 0 ? C::R * C::WARPS : 1];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const bool keep = slot[i] >= 0 && slot[i] < a.num_slots;
    if (!keep && slot[i] != -1 && u == 0 && head[i] == 0) set_dev_err(a.dev_err, PA_DEV_ERR_SLOT);
    const int64_t at = (slot[i] * heads + head[i]) * D;
    if constexpr (FMT == 0) {
      if (keep) {
        uint16_t* row = static_cast<uint16_t*>(cache) + at;
        st_vec8(row + p.va, xa[i], true);
        st_vec8(row + p.vb, xb[i], true);
      }
    } else {
      const float scale = quantise_unit<D, F16, FMT>(
          xa[i], xb[i], p, static_cast<unsigned char*>(cache) + at, keep);
      if (u == 0) row_scales[warp * C::R + i * C::HPW + lane / C::UNITS] = scale;
    }
  }
  if constexpr (FMT != 0) {
    // scales together, as above
    __syncthreads();
    for (uint32_t n = threadIdx.x; n < tokens * heads; n += blockDim.x) {
      const uint32_t h = n / tokens, t = tok0 + (n - h * tokens);
      const uint32_t r = t * heads + h - row0;  // (wraps below the block's first row)
      if (r >= rows || r >= total - row0) continue;
      const int32_t s = __ldg(a.slots + t);
      if (s >= 0 && s < a.num_slots)
        write_scale(is_v ? a.v_scale : a.k_scale, s, heads, (int)h, a.block_size, row_scales[r]);
    }
  }
}

// FMT: 0 = 16-bit cache, else a pa_q8_format. Blocks of wide items come first, then (FLAT) flat
// blocks of queries, keys and values (RowsArgs). The form without flat blocks has no shared
// memory for their angles and fewer registers.
template <int D, bool F16, int FMT, bool ROT, bool ADJ, bool FLAT>
__global__ void __launch_bounds__(kRowsThreads, ROT ? 5 : FLAT ? 6 : 8)
    kv_rows_kernel(const RowsArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  if constexpr (FLAT) {
    uint32_t blk = blockIdx.x;
    if (blk >= a.wide_blocks) {
      blk -= a.wide_blocks;
      const bool is_q = ROT && blk < a.q_blocks;
      if (ROT && !is_q) blk -= a.q_blocks;
      const bool is_v = !is_q && blk >= a.kv_blocks;
      if (is_v) blk -= a.kv_blocks;
      flat_rows<D, F16, FMT, ROT, ADJ>(a, blk, is_q, is_v);
      return;
    }
  }
  if constexpr (ROT || !FLAT) wide_rows<D, F16, FMT, ROT, ADJ>(a);
}

template <int D, bool F16, int FMT, bool ROT, bool ADJ>
int launch_rows_t(RowsArgs a, const DeviceInfo& info, cudaStream_t stream) {
  constexpr int64_t R = RowsCfg<D>::R;
  auto over = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  const int64_t n = a.num_tokens, q_heads = ROT ? a.num_heads : 0, kv_heads = a.num_kv_heads;
  // Wide items have to be half full (of 128 dims: more than that; 20,000 tokens of 4 / 4 heads 24.7 us
  // flat, 29.0 wide, of 6 / 6 32.4 and 31.0), queries three quarters where keys and values take
  // flat blocks anyway (32,000 of 4 / 2 heads 26.1 and 30.4, of 9 / 3 42.8 and 50.6). Without
  // angles only full ones are wide (20,000 of 12 heads of 64 15.8 and 18.0). The 8-bit rotary form
  // follows the 16-bit one's rule, which serves it less well: 17,556 tokens to e4m3 and int8 take, of
  // 16 / 8 heads of 128, 43.8, 45.6 us wide and 47.5, 49.0 flat, of 4 / 4 30.1, 33.1 and 21.0, 22.3;
  // but of 6 / 6 31.2, 34.1 and 30.2, 31.8, of 12 / 12 58.6, 63.7 and 54.3, 57.1, of 32 / 8 heads
  // of 64 41.5, 43.9 and 38.2, 39.1.
  const bool kv_wide =
      ROT ? (D == 128 ? 2 * kv_heads > R : 2 * kv_heads >= R) : kv_heads % R == 0;
  const bool q_wide = kv_wide ? 2 * q_heads >= R : 4 * q_heads >= 3 * over(q_heads, R) * R;
  a.q_chunks = q_wide ? (int)over(q_heads, R) : 0;
  a.kv_chunks = kv_wide ? (int)over(kv_heads, R) : 0;
  const int64_t chunks = a.q_chunks + 2 * (int64_t)a.kv_chunks;
  // (2^31 rows are more memory than there is)
  if (n * q_heads > INT32_MAX || n * kv_heads > INT32_MAX || n * chunks > INT32_MAX ||
      (q_heads + R) * D > INT32_MAX || (kv_heads + R) * D > INT32_MAX)
    return PA_ERR_UNSUPPORTED;
  const int64_t q_items = q_wide ? 0 : over(n * q_heads, R);
  const int64_t kv_items = kv_wide ? 0 : over(n * kv_heads, R);
  // few items are spread over the SMs in blocks of two warps
  const int threads =
      n * chunks + q_items + 2 * kv_items < (int64_t)info.num_sms * 8 ? 64 : kRowsThreads;
  const int warps = threads / 32;
  const int64_t wide = FMT == 0 ? over(n * chunks, warps) : over(n, warps) * chunks;
  const int64_t q_flat = over(q_items, warps), kv_flat = over(kv_items, warps);
  const int64_t blocks = wide + q_flat + 2 * kv_flat;
  if (blocks > INT32_MAX) return PA_ERR_UNSUPPORTED;
  a.wide_blocks = (uint32_t)wide;
  a.q_blocks = (uint32_t)q_flat;
  a.kv_blocks = (uint32_t)kv_flat;
  // ceil(2^64 / heads): the high half of its product with r is r / heads (0 for one head)
  auto magic = [](int64_t heads) { return heads > 1 ? UINT64_MAX / (uint64_t)heads + 1 : 0; };
  a.q_magic = magic(q_heads);
  a.kv_magic = magic(kv_heads);
  const bool flat = q_flat + kv_flat > 0;
  const cudaError_t rc =
      flat ? launch_dependent(kv_rows_kernel<D, F16, FMT, ROT, ADJ, true>, dim3((unsigned)blocks),
                              dim3((unsigned)threads), 0, stream, a)
           : launch_dependent(kv_rows_kernel<D, F16, FMT, ROT, ADJ, false>, dim3((unsigned)blocks),
                              dim3((unsigned)threads), 0, stream, a);
  if (rc != cudaSuccess) return PA_ERR_CUDA;
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
