// store_q8.cu — pa_store_kvcache_q8 (kv_rows.cuh) and pa_load_kvcache_q8.
#include "kv_rows.cuh"

namespace pa {

int launch_store_rows(const RowsArgs& a, int fmt, int head_dim, bool f16, const DeviceInfo& info,
                      cudaStream_t stream) {
  const bool e4m3 = fmt == PA_Q8_E4M3;
  if (head_dim == 128) {
    if (f16)
      return e4m3 ? launch_rows_t<128, true, PA_Q8_E4M3, false, false>(a, info, stream)
                  : launch_rows_t<128, true, PA_Q8_INT8, false, false>(a, info, stream);
    return e4m3 ? launch_rows_t<128, false, PA_Q8_E4M3, false, false>(a, info, stream)
                : launch_rows_t<128, false, PA_Q8_INT8, false, false>(a, info, stream);
  }
  if (f16)
    return e4m3 ? launch_rows_t<64, true, PA_Q8_E4M3, false, false>(a, info, stream)
                : launch_rows_t<64, true, PA_Q8_INT8, false, false>(a, info, stream);
  return e4m3 ? launch_rows_t<64, false, PA_Q8_E4M3, false, false>(a, info, stream)
              : launch_rows_t<64, false, PA_Q8_INT8, false, false>(a, info, stream);
}

int launch_rotary_d64_bf16(const RowsArgs& a, int fmt, const DeviceInfo& info, cudaStream_t stream);
int launch_rotary_d64_f16(const RowsArgs& a, int fmt, const DeviceInfo& info, cudaStream_t stream);
int launch_rotary_d128_bf16(const RowsArgs& a, int fmt, const DeviceInfo& info,
                            cudaStream_t stream);
int launch_rotary_d128_f16(const RowsArgs& a, int fmt, const DeviceInfo& info, cudaStream_t stream);

int launch_rotary_rows(const RowsArgs& a, int fmt, int head_dim, bool f16, const DeviceInfo& info,
                       cudaStream_t stream) {
  if (head_dim == 128)
    return f16 ? launch_rotary_d128_f16(a, fmt, info, stream)
               : launch_rotary_d128_bf16(a, fmt, info, stream);
  return f16 ? launch_rotary_d64_f16(a, fmt, info, stream)
             : launch_rotary_d64_bf16(a, fmt, info, stream);
}

namespace {

constexpr int kLoadThreads = 256;
constexpr int kLoadUnroll = 4;  // row groups a warp loads before it uses the first

// A block's rows (token, KV head) are consecutive; a lane holds 8 codes, D/8 lanes a row, so that
// every store of the warp covers 512 consecutive bytes (with 16 codes a lane writes half a
// sector at a time: 46.1 us against 36.9 for 150 blocks of 256 x 8 x 128 e4m3, 6.4 TB/s or 0.94 of
// the copy rate; 1,000 blocks 231 us, 1.01). A warp takes kLoadUnroll consecutive groups of
// 32 / (D/8) rows of K or V of one listed block.
template <int D, bool F16, int FMT>
__global__ void __launch_bounds__(kLoadThreads)
    load_q8_kernel(const LoadQ8Args a, const int parts, const uint64_t per_head) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = kLoadUnroll;
  const int lane = threadIdx.x & 31;
  const int rows = a.block_size * a.num_kv_heads;
  const int64_t item = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  pdl_launch_dependents();
  pdl_wait();
  if (item >= (int64_t)a.num_listed * 2 * parts) return;
  const int64_t which = item / parts;  // 2 i: K of listed block i, 2 i + 1: its V
  const int r0 = (int)(item - which * parts) * (RPW * U) + lane / LPR;
  const bool v = (which & 1) != 0;
  const int blk = __ldg(a.blocks + (which >> 1));
  if (blk < 0 || blk >= a.num_blocks) {
    if (blk != -1 && lane == 0) set_dev_err(a.dev_err, PA_DEV_ERR_BLOCK_ID);
    return;
  }
  const unsigned char* src = static_cast<const unsigned char*>(v ? a.v_codes : a.k_codes) +
                             (int64_t)blk * rows * D + lane % LPR * 8;
  uint16_t* dst = static_cast<uint16_t*>(v ? a.v_out : a.k_out) + (which >> 1) * rows * D +
                  lane % LPR * 8;
  const float* scales = (v ? a.v_scale : a.k_scale) + (int64_t)blk * rows;
  uint2 w[U];
  float sc[U];
  // (not under a condition, which would put each load next to its use: 42.1 us with int8)
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int r = min(r0 + i * RPW, rows - 1);
    w[i] = __ldg(reinterpret_cast<const uint2*>(src + (int64_t)r * D));
    // r / num_kv_heads
    const uint32_t t = per_head ? (uint32_t)__umul64hi((uint64_t)r, per_head) : (uint32_t)r;
    sc[i] = __ldg(scales + (r - t * a.num_kv_heads) * a.block_size + t);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int r = r0 + i * RPW;
    if (r < rows) {
      const uint32_t p[2] = {w[i].x, w[i].y};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[4];
        widen4_f32<FMT>(p[e], x);
        o[2 * e] = narrow2<F16>(x[0] * sc[i], x[1] * sc[i]);
        o[2 * e + 1] = narrow2<F16>(x[2] * sc[i], x[3] * sc[i]);
      }
      *reinterpret_cast<uint4*>(dst + (int64_t)r * D) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int D, bool F16, int FMT>
int launch_load_t(const LoadQ8Args& a, const DeviceInfo& info, cudaStream_t stream) {
  constexpr int per_item = 32 / (D / 8) * kLoadUnroll;
  const int parts = (a.block_size * a.num_kv_heads + per_item - 1) / per_item;
  const int64_t items = (int64_t)a.num_listed * 2 * parts;
  // ceil(2^64 / heads): the high half of its product with r is r / heads for every 32-bit r and
  // heads > 1 (0 for one head)
  const uint64_t heads = (uint64_t)a.num_kv_heads;
  const uint64_t per_head = heads > 1 ? UINT64_MAX / heads + 1 : 0;
  // few items are spread over the SMs in blocks of two warps
  const int threads = items < (int64_t)info.num_sms * 8 ? 64 : kLoadThreads;
  const int64_t blocks = (items + threads / 32 - 1) / (threads / 32);
  if (blocks > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (launch_dependent(load_q8_kernel<D, F16, FMT>, dim3((unsigned)blocks), dim3((unsigned)threads),
                       0, stream, a, parts, per_head) != cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D, bool F16>
int launch_load_fmt(const LoadQ8Args& a, int fmt, const DeviceInfo& info, cudaStream_t stream) {
  return fmt == PA_Q8_E4M3 ? launch_load_t<D, F16, PA_Q8_E4M3>(a, info, stream)
                           : launch_load_t<D, F16, PA_Q8_INT8>(a, info, stream);
}

}  // namespace

int launch_load_q8(const LoadQ8Args& a, int fmt, int head_dim, bool f16, const DeviceInfo& info,
                   cudaStream_t stream) {
  if (head_dim == 128)
    return f16 ? launch_load_fmt<128, true>(a, fmt, info, stream)
               : launch_load_fmt<128, false>(a, fmt, info, stream);
  return f16 ? launch_load_fmt<64, true>(a, fmt, info, stream)
             : launch_load_fmt<64, false>(a, fmt, info, stream);
}

}  // namespace pa
