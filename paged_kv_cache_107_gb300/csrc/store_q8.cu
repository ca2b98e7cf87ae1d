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
constexpr int kLoadUnroll = 4;       // row groups a warp loads before it uses the first
constexpr int kLoadBlocksPerSM = 4;  // resident blocks per SM (register budget)

// A block's rows (token, KV head) are consecutive; a lane holds 16 codes, D/16 lanes a row. A
// warp takes kLoadUnroll consecutive groups of 32 / (D/16) rows of K or V of one listed block:
// 512 bytes of codes in and 1,024 of elements out for each group.
template <int D, bool F16, int FMT>
__global__ void __launch_bounds__(kLoadThreads, kLoadBlocksPerSM)
    load_q8_kernel(const LoadQ8Args a, const int parts) {
  constexpr int UNITS = D / 16, RPW = 32 / UNITS, U = kLoadUnroll;
  const int lane = threadIdx.x & 31;
  const int u = lane % UNITS, rl = lane / UNITS;
  const int rows = a.block_size * a.num_kv_heads;
  const int64_t items = (int64_t)a.num_listed * 2 * parts;
  const int64_t warps = (int64_t)gridDim.x * (kLoadThreads / 32);
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t item = (int64_t)blockIdx.x * (kLoadThreads / 32) + (threadIdx.x >> 5);
       item < items; item += warps) {
    const int part = (int)(item % parts);
    const int kv = (int)(item / parts & 1);
    const int64_t at = item / parts >> 1;
    const int blk = __ldg(a.blocks + at);
    if (blk < 0 || blk >= a.num_blocks) {
      if (blk != -1 && lane == 0) set_dev_err(a.dev_err, PA_DEV_ERR_BLOCK_ID);
      continue;
    }
    const unsigned char* src =
        static_cast<const unsigned char*>(kv ? a.v_codes : a.k_codes) + (int64_t)blk * rows * D;
    uint16_t* dst = static_cast<uint16_t*>(kv ? a.v_out : a.k_out) + at * rows * D;
    const float* scales = (kv ? a.v_scale : a.k_scale) + (int64_t)blk * rows;
    const int r0 = part * (RPW * U) + rl;
    uint4 w[U];
    float sc[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = r0 + i * RPW;
      if (r < rows) {
        w[i] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)r * D + u * 16));
        const uint32_t t = (uint32_t)r / (uint32_t)a.num_kv_heads;
        sc[i] = __ldg(scales + (r - t * a.num_kv_heads) * a.block_size + t);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = r0 + i * RPW;
      if (r < rows) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(&w[i]);
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t lo, hi;
          widen4<FMT, false>(p[e], lo, hi);
          const float2 x = f16x2_f2(lo), y = f16x2_f2(hi);
          o[2 * e] = narrow2<F16>(x.x * sc[i], x.y * sc[i]);
          o[2 * e + 1] = narrow2<F16>(y.x * sc[i], y.y * sc[i]);
        }
        uint4* q = reinterpret_cast<uint4*>(dst + (int64_t)r * D + u * 16);
        q[0] = make_uint4(o[0], o[1], o[2], o[3]);
        q[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

template <int D, bool F16, int FMT>
int launch_load_t(const LoadQ8Args& a, const DeviceInfo& info, cudaStream_t stream) {
  constexpr int per_item = 32 / (D / 16) * kLoadUnroll;
  const int parts = (a.block_size * a.num_kv_heads + per_item - 1) / per_item;
  const int64_t items = (int64_t)a.num_listed * 2 * parts;
  int64_t blocks = (items + kLoadThreads / 32 - 1) / (kLoadThreads / 32);
  const int64_t cap = (int64_t)info.num_sms * kLoadBlocksPerSM;  // one resident wave
  if (blocks > cap) blocks = cap;
  if (launch_dependent(load_q8_kernel<D, F16, FMT>, dim3((unsigned)blocks), dim3(kLoadThreads), 0,
                       stream, a, parts) != cudaSuccess)
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
