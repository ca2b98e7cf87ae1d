// pa_api.cu — the exported C ABI (include/pa.h): argument validation, then launch.
// Nothing here allocates device memory or synchronises the host.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "../../include/pa.h"
#include "pa_launch.h"

namespace pa {

bool current_device_info(DeviceInfo* info) {
  static DeviceInfo cache[64];
  static bool valid[64] = {false};
  static std::mutex mu;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (!valid[dev]) {
    DeviceInfo d{};
    d.device = dev;
    if (cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return false;
    cache[dev] = d;
    valid[dev] = true;
  }
  *info = cache[dev];
  return true;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

constexpr float kLog2e = 1.4426950408889634f;  // exp(x) = exp2(x * log2(e))

static float natural_scale(float scale, int head_dim) {
  if (!(scale > 0.f) || isnan(scale)) scale = 1.0f / sqrtf((float)head_dim);
  return scale;
}
static float resolve_scale(float scale, int head_dim) {
  return natural_scale(scale, head_dim) * kLog2e;
}

// Checks pa_score_mod and folds its factors (ScoreModArgs).
static int resolve_mod(const pa_score_mod* mod, float scale, int head_dim, ScoreModArgs* m) {
  if (!mod) return PA_ERR_NULL;
  if (!(mod->softcap >= 0.f) || isinf(mod->softcap) || mod->window < 0 || mod->sink < 0)
    return PA_ERR_SHAPE;
  if (head_dim <= 0) return PA_ERR_UNSUPPORTED;
  m->cap2 = mod->softcap * kLog2e;
  m->cap_in = mod->softcap > 0.f ? natural_scale(scale, head_dim) / mod->softcap : 0.f;
  // (below FLT_MIN the quotient loses bits, to the last one)
  if (isinf(m->cap2) || isinf(m->cap_in) || (m->cap2 > 0.f && m->cap_in < FLT_MIN))
    return PA_ERR_SHAPE;
  const double z = (double)m->cap_in * m->cap_in;
  double f = (double)m->cap2 * m->cap_in;
  for (int i = 0; i < 6; ++i, f *= z) {
    m->poly[i][0] = m->poly[i][1] = (float)(f * kTanhPoly[i]);
    if (i < 4) m->poly3[i][0] = m->poly3[i][1] = (float)(f * kTanhPoly3[i]);
  }
  m->z_lim = z > 0 ? (float)(1.0 / z) : 0.f;
  m->z_lim3 = z > 0 ? (float)(0.36 / z) : 0.f;
  // A cap so small that a coefficient leaves fp32 (inf * 0 for a zero product): no product but
  // zero is in the polynomials' range, and every tile takes the exact way.
  if (isinf(m->poly[5][0])) {
    for (int i = 0; i < 6; ++i) m->poly[i][0] = m->poly[i][1] = 0.f;
    for (int i = 0; i < 4; ++i) m->poly3[i][0] = m->poly3[i][1] = 0.f;
    m->z_lim = m->z_lim3 = 0.f;
  }
  m->slopes = mod->slopes;
  m->window = mod->window;
  m->sink = mod->sink;
  m->prefix_lens = mod->prefix_lens;
  return PA_OK;
}

}  // namespace pa

extern "C" {

const char* pa_status_str(int status) {
  switch (status) {
    case PA_OK: return "PA_OK";
    case PA_ERR_NULL: return "PA_ERR_NULL: a required pointer is NULL";
    case PA_ERR_SHAPE: return "PA_ERR_SHAPE: inconsistent sizes";
    case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED: head_dim, group size or block size not supported";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE: decode workspace missing or too small";
    case PA_ERR_CUDA: return "PA_ERR_CUDA: CUDA runtime error";
    case PA_ERR_ALIGN: return "PA_ERR_ALIGN: pointer or stride not 16-byte aligned";
    default: return "unknown pa status";
  }
}

int pa_version(void) { return (1 << 16) | 0; }

int pa_store_kvcache(const void* k, const void* v, int64_t k_tok_stride, int64_t v_tok_stride,
                     void* k_cache, void* v_cache, const int32_t* slot_mapping, int num_tokens,
                     int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                     int* dev_err, void* stream) {
  if (num_tokens < 0 || num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0)
    return PA_ERR_SHAPE;
  if (!pa::head_dim_supported(head_dim)) return PA_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  if (k_tok_stride < row || v_tok_stride < row) return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !k_cache || !v_cache || !slot_mapping) return PA_ERR_NULL;
  pa::DeviceInfo info;
  if (!pa::current_device_info(&info)) return PA_ERR_CUDA;
  return pa::launch_store_kvcache(k, v, k_tok_stride, v_tok_stride, k_cache, v_cache,
                                  slot_mapping, num_tokens, num_kv_heads, head_dim,
                                  num_blocks * (int64_t)block_size, dev_err,
                                  static_cast<cudaStream_t>(stream), info.num_sms);
}

int pa_staged_write_apply(void* base, int64_t num_rows, int64_t num_cols, int64_t row_stride,
                          int elem_bytes, const int32_t* rows, const int32_t* starts,
                          const int32_t* offsets, const void* values, int num_writes,
                          int64_t num_values, int* dev_err, void* stream) {
  if (num_rows < 0 || num_cols < 0 || row_stride < num_cols || num_writes < 0 || num_values < 0)
    return PA_ERR_SHAPE;
  if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4 && elem_bytes != 8)
    return PA_ERR_UNSUPPORTED;
  if (num_values > INT32_MAX) return PA_ERR_UNSUPPORTED;  // offsets are int32
  if (num_values == 0) return PA_OK;
  if (num_writes == 0) return PA_ERR_SHAPE;  // values without a run to hold them
  if (!base || !rows || !starts || !offsets || !values) return PA_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(values)) %
          (uintptr_t)elem_bytes !=
      0)
    return PA_ERR_ALIGN;
  pa::DeviceInfo info;
  if (!pa::current_device_info(&info)) return PA_ERR_CUDA;
  return pa::launch_staged_write(base, num_rows, num_cols, row_stride, elem_bytes, rows, starts,
                                 offsets, values, num_writes, num_values, dev_err,
                                 static_cast<cudaStream_t>(stream), info.num_sms);
}

int pa_staged_upload_apply(void* base, int64_t num_rows, int64_t num_cols, int64_t row_stride,
                           int elem_bytes, const void* packed_host, void* packed_dev,
                           const pa_staged_layout* layout, int* dev_err, void* stream) {
  if (!layout) return PA_ERR_NULL;
  if (num_rows < 0 || num_cols < 0 || row_stride < num_cols || layout->bytes < 0 ||
      layout->num_writes < 0 || layout->num_values < 0)
    return PA_ERR_SHAPE;
  if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4 && elem_bytes != 8)
    return PA_ERR_UNSUPPORTED;
  if (layout->bytes == 0) return PA_OK;
  if (!packed_host || !packed_dev || (layout->num_values > 0 && !base)) return PA_ERR_NULL;
  if (layout->num_values > 0 && layout->num_writes == 0) return PA_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(packed_dev) & 15) ||
      (reinterpret_cast<uintptr_t>(base) % (uintptr_t)elem_bytes) ||
      (layout->values_offset % 16) || (layout->rows_offset % 4) || (layout->starts_offset % 4) ||
      (layout->offsets_offset % 4))
    return PA_ERR_ALIGN;
  pa::DeviceInfo info;
  if (!pa::current_device_info(&info)) return PA_ERR_CUDA;
  return pa::launch_staged_upload_apply(base, num_rows, num_cols, row_stride, elem_bytes,
                                        packed_host, packed_dev, layout, dev_err,
                                        static_cast<cudaStream_t>(stream), info.num_sms);
}

size_t pa_sample_workspace_size(int num_seqs) {
  if (num_seqs < 0) return 0;
  return pa::sample_workspace_bytes(num_seqs > 0 ? num_seqs : 1);
}

int pa_gumbel_sample(int64_t* out, const void* logits, int64_t row_stride, int logits_dtype,
                     int num_seqs, int vocab_size, const float* temperatures,
                     const uint64_t* seeds, const uint64_t* offsets, void* workspace,
                     size_t workspace_bytes, int* dev_err, void* stream) {
  if (num_seqs < 0 || vocab_size <= 0 || row_stride < vocab_size) return PA_ERR_SHAPE;
  if (logits_dtype != PA_DTYPE_F32 && logits_dtype != PA_DTYPE_BF16) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!out || !logits || !temperatures || !seeds || !offsets) return PA_ERR_NULL;
  if (!workspace || workspace_bytes < pa::sample_workspace_bytes(num_seqs))
    return PA_ERR_WORKSPACE;
  const uintptr_t esz = logits_dtype == PA_DTYPE_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(logits) % esz) || (reinterpret_cast<uintptr_t>(out) & 7) ||
      (reinterpret_cast<uintptr_t>(seeds) & 7) || (reinterpret_cast<uintptr_t>(offsets) & 7) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return PA_ERR_ALIGN;
  pa::DeviceInfo info;
  if (!pa::current_device_info(&info)) return PA_ERR_CUDA;
  return pa::launch_gumbel_sample(out, logits, row_stride, logits_dtype == PA_DTYPE_BF16,
                                  num_seqs, vocab_size, temperatures, seeds, offsets, workspace,
                                  dev_err, static_cast<cudaStream_t>(stream), info.num_sms);
}

size_t pa_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim) {
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || !pa::head_dim_supported(head_dim))
    return 0;
  pa::DeviceInfo info;
  if (!pa::current_device_info(&info)) return 0;
  size_t a, b, c, total;
  pa::decode_workspace_layout(num_seqs, num_heads, num_kv_heads, pa::decode_max_ctas(info), &a,
                              &b, &c, &total);
  return total;
}

}  // extern "C"

namespace pa {

int decode_prepare(void* out, const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* context_lens, int num_seqs, int num_heads, int num_kv_heads,
                   int head_dim, int dtype, int block_size, int64_t num_blocks, float scale,
                   int grid_ctas, int* dev_err, const DecodeStepInput* step, DecodeArgs* a,
                   DeviceInfo* info, bool* nothing) {
  *nothing = false;
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || block_size <= 0 ||
      num_blocks <= 0 || max_blocks_per_seq < 0 || grid_ctas < 0)
    return PA_ERR_SHAPE;
  if (num_heads % num_kv_heads != 0) return PA_ERR_SHAPE;
  if (!head_dim_supported(head_dim) || !decode_supported(num_heads, num_kv_heads) ||
      (dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_F16))
    return PA_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (step) {
    const int64_t row = (int64_t)num_kv_heads * head_dim;
    if (step->k_new_stride < row || step->v_new_stride < row) return PA_ERR_SHAPE;
  }
  if (num_seqs == 0) {
    *nothing = true;
    return PA_OK;
  }
  if (step) {
    if (!step->k_new || !step->v_new || !step->slot_mapping) return PA_ERR_NULL;
    // rows move with bulk copies: 16-byte aligned starts
    if (!aligned16(step->k_new) || !aligned16(step->v_new) || (step->k_new_stride & 7) ||
        (step->v_new_stride & 7))
      return PA_ERR_ALIGN;
  }
  if (!out || !q || !k_cache || !v_cache || !context_lens) return PA_ERR_NULL;
  if (max_blocks_per_seq > 0 && !block_tables) return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_ALIGN;
  if (!current_device_info(info)) return PA_ERR_CUDA;
  const bool auto_grid = grid_ctas == 0;
  if (auto_grid) grid_ctas = info->num_sms;
  if (grid_ctas > decode_max_ctas(*info)) return PA_ERR_SHAPE;
  *a = DecodeArgs{};
  a->out = out;
  a->q = q;
  a->k_cache = k_cache;
  a->v_cache = v_cache;
  a->block_tables = block_tables;
  a->context_lens = context_lens;
  a->max_blocks = max_blocks_per_seq;
  a->num_seqs = num_seqs;
  a->num_heads = num_heads;
  a->num_kv_heads = num_kv_heads;
  a->block_size = block_size;
  a->num_blocks = num_blocks;
  a->scale_log2 = resolve_scale(scale, head_dim);
  a->head_dim = head_dim;
  a->f16 = dtype == PA_DTYPE_F16;
  a->grid_ctas = grid_ctas;
  a->min_tiles = auto_grid ? kDecodeMinTilesPerCta : 1;
  a->dev_err = dev_err;
  if (step) {
    a->k_new = step->k_new;
    a->v_new = step->v_new;
    a->k_new_stride = step->k_new_stride;
    a->v_new_stride = step->v_new_stride;
    a->slot_mapping = step->slot_mapping;
  }
  return PA_OK;
}

size_t decode_bind_workspace(DecodeArgs* a, unsigned char* ws, int layout_ctas) {
  size_t off_c, off_l, off_o, total;
  decode_workspace_layout(a->num_seqs, a->num_heads, a->num_kv_heads, layout_ctas, &off_c,
                          &off_l, &off_o, &total);
  a->counters = ws ? reinterpret_cast<int*>(ws + off_c) : nullptr;
  a->part_lse = ws ? reinterpret_cast<float*>(ws + off_l) : nullptr;
  a->part_o = ws ? reinterpret_cast<float*>(ws + off_o) : nullptr;
  return total;
}

// Binds the caller's workspace, laid out for the largest grid the device allows (so one
// workspace serves every grid_ctas).
static int decode_check_workspace(DecodeArgs* a, const DeviceInfo& info, void* workspace,
                                  size_t workspace_bytes) {
  const size_t need =
      decode_bind_workspace(a, static_cast<unsigned char*>(workspace), decode_max_ctas(info));
  if (!workspace || workspace_bytes < need) return PA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return PA_ERR_ALIGN;
  return PA_OK;
}

// Points the scratch of pa_decode_shared into `ws` (may be null: only the size is wanted);
// returns the bytes needed. Nothing in it outlives a call.
static size_t shared_bind_workspace(DecodeSharedArgs* a, unsigned char* ws) {
  size_t at = 0;
  auto take = [&](auto** p, size_t n) {
    using T = std::remove_reference_t<decltype(**p)>;
    *p = ws ? reinterpret_cast<T*>(ws + at) : nullptr;
    at += (n * sizeof(T) + 255) & ~size_t(255);
  };
  const size_t rows = (size_t)a->num_seqs * a->num_heads;
  const size_t more = (size_t)a->grid_ctas * 256;
  const size_t cut = (size_t)a->grid_ctas * a->num_heads;
  take(&a->sh.more_o, more * a->head_dim);
  take(&a->sh.more_lse, more);
  take(&a->part_o, cut * a->head_dim);
  take(&a->part_lse, cut);
  take(&a->sh.first_o, rows * a->head_dim);
  take(&a->sh.first_lse, rows);
  take(&a->sh.rest_o, rows * a->head_dim);
  take(&a->sh.rest_lse, rows);
  take(&a->sh.prefix, (size_t)a->num_seqs * a->num_kv_heads);
  take(&a->sh.rest, (size_t)a->num_seqs);
  return at;
}

// pa_decode and pa_decode_step; `step` is null for the plain call.
static int decode_entry(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_tables, int max_blocks_per_seq,
                        const int32_t* context_lens, int num_seqs, int num_heads,
                        int num_kv_heads, int head_dim, int dtype, int block_size,
                        int64_t num_blocks, float scale, int grid_ctas, void* workspace,
                        size_t workspace_bytes, int* dev_err, void* stream,
                        const DecodeStepInput* step) {
  DecodeArgs a;
  DeviceInfo info;
  bool nothing = false;
  const int rc = decode_prepare(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                context_lens, num_seqs, num_heads, num_kv_heads, head_dim,
                                dtype, block_size, num_blocks, scale, grid_ctas, dev_err, step,
                                &a, &info, &nothing);
  if (rc != PA_OK || nothing) return rc;
  const int wrc = decode_check_workspace(&a, info, workspace, workspace_bytes);
  if (wrc != PA_OK) return wrc;
  if (step) return launch_decode_step(a, info, static_cast<cudaStream_t>(stream));
  return launch_decode(a, info, static_cast<cudaStream_t>(stream));
}

}  // namespace pa

namespace pa {

// pa_prefill_varlen and pa_prefill_mod: argument validation and packing. On PA_OK, *nothing
// is set when there is no query to launch for.
static int prefill_prepare(void* out, const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, int max_blocks_per_seq,
                           const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                           int num_seqs, int max_seqlen_q, int max_seqlen_k, int num_heads,
                           int num_kv_heads, int head_dim, int dtype, int block_size,
                           int64_t num_blocks, int causal, float scale, int* dev_err,
                           PrefillArgs* a, DeviceInfo* info, bool* nothing) {
  *nothing = false;
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || block_size <= 0 ||
      num_blocks <= 0 || max_blocks_per_seq < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return PA_ERR_SHAPE;
  if (num_heads % num_kv_heads != 0) return PA_ERR_SHAPE;
  if (!head_dim_supported(head_dim) ||
      !prefill_supported(num_heads, num_kv_heads, block_size) ||
      (dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_F16))
    return PA_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (max_seqlen_k > (int64_t)max_blocks_per_seq * block_size) return PA_ERR_SHAPE;
  if (num_seqs == 0 || max_seqlen_q == 0) {
    *nothing = true;
    return PA_OK;
  }
  if (!out || !q || !k_cache || !v_cache || !cu_seqlens_q || !cu_seqlens_k) return PA_ERR_NULL;
  if (max_blocks_per_seq > 0 && !block_tables) return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) ||
      !aligned16(v_cache))
    return PA_ERR_ALIGN;
  if (!current_device_info(info)) return PA_ERR_CUDA;
  a->out = out;
  a->q = q;
  a->k_cache = k_cache;
  a->v_cache = v_cache;
  a->block_tables = block_tables;
  a->cu_seqlens_q = cu_seqlens_q;
  a->cu_seqlens_k = cu_seqlens_k;
  a->max_blocks = max_blocks_per_seq;
  a->num_seqs = num_seqs;
  a->max_seqlen_q = max_seqlen_q;
  a->max_seqlen_k = max_seqlen_k;
  a->num_heads = num_heads;
  a->num_kv_heads = num_kv_heads;
  a->block_size = block_size;
  a->num_blocks = num_blocks;
  a->causal = causal ? 1 : 0;
  a->scale_log2 = resolve_scale(scale, head_dim);
  a->head_dim = head_dim;
  a->f16 = dtype == PA_DTYPE_F16;
  a->dev_err = dev_err;
  return PA_OK;
}

}  // namespace pa

extern "C" {

int pa_decode(void* out, const void* q, const void* k_cache, const void* v_cache,
              const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
              int num_seqs, int num_heads, int num_kv_heads, int head_dim, int dtype,
              int block_size, int64_t num_blocks, float scale, int grid_ctas, void* workspace,
              size_t workspace_bytes, int* dev_err, void* stream) {
  return pa::decode_entry(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                          context_lens, num_seqs, num_heads, num_kv_heads, head_dim, dtype,
                          block_size, num_blocks, scale, grid_ctas, workspace, workspace_bytes,
                          dev_err, stream, nullptr);
}

int pa_decode_step(void* out, const void* q, const void* k_new, const void* v_new,
                   int64_t k_new_stride, int64_t v_new_stride, void* k_cache, void* v_cache,
                   const int32_t* slot_mapping, const int32_t* block_tables,
                   int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                   int num_heads, int num_kv_heads, int head_dim, int dtype, int block_size,
                   int64_t num_blocks, float scale, int grid_ctas, void* workspace,
                   size_t workspace_bytes, int* dev_err, void* stream) {
  const pa::DecodeStepInput step{k_new, v_new, k_new_stride, v_new_stride, slot_mapping};
  return pa::decode_entry(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                          context_lens, num_seqs, num_heads, num_kv_heads, head_dim, dtype,
                          block_size, num_blocks, scale, grid_ctas, workspace, workspace_bytes,
                          dev_err, stream, &step);
}

int pa_prefill_varlen(void* out, const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, int max_blocks_per_seq,
                      const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int num_seqs,
                      int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                      int head_dim, int dtype, int block_size, int64_t num_blocks, int causal,
                      float scale, int* dev_err, void* stream) {
  pa::PrefillArgs a;
  pa::DeviceInfo info;
  bool nothing = false;
  const int rc = pa::prefill_prepare(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                     cu_seqlens_q, cu_seqlens_k, num_seqs, max_seqlen_q,
                                     max_seqlen_k, num_heads, num_kv_heads, head_dim, dtype,
                                     block_size, num_blocks, causal, scale, dev_err, &a, &info,
                                     &nothing);
  if (rc != PA_OK || nothing) return rc;
  return pa::launch_prefill(a, info, static_cast<cudaStream_t>(stream));
}

int pa_decode_mod(void* out, const void* q, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, int max_blocks_per_seq,
                  const int32_t* context_lens, int num_seqs, int num_heads, int num_kv_heads,
                  int head_dim, int dtype, int block_size, int64_t num_blocks, float scale,
                  const pa_score_mod* mod, int grid_ctas, void* workspace,
                  size_t workspace_bytes, int* dev_err, void* stream) {
  pa::DecodeModArgs a;
  pa::DeviceInfo info;
  bool nothing = false;
  int rc = pa::resolve_mod(mod, scale, head_dim, &a.mod);
  if (rc != PA_OK) return rc;
  rc = pa::decode_prepare(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                          context_lens, num_seqs, num_heads, num_kv_heads, head_dim, dtype,
                          block_size, num_blocks, scale, grid_ctas, dev_err, nullptr, &a, &info,
                          &nothing);
  if (rc != PA_OK || nothing) return rc;
  rc = pa::decode_check_workspace(&a, info, workspace, workspace_bytes);
  if (rc != PA_OK) return rc;
  return pa::launch_decode_mod(a, info, static_cast<cudaStream_t>(stream));
}

int pa_prefill_mod(void* out, const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int num_seqs,
                   int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                   int head_dim, int dtype, int block_size, int64_t num_blocks, int causal,
                   float scale, const pa_score_mod* mod, int* dev_err, void* stream) {
  pa::PrefillModArgs a;
  pa::DeviceInfo info;
  bool nothing = false;
  int rc = pa::resolve_mod(mod, scale, head_dim, &a.mod);
  if (rc != PA_OK) return rc;
  rc = pa::prefill_prepare(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                           cu_seqlens_q, cu_seqlens_k, num_seqs, max_seqlen_q, max_seqlen_k,
                           num_heads, num_kv_heads, head_dim, dtype, block_size, num_blocks,
                           causal, scale, dev_err, &a, &info, &nothing);
  if (rc != PA_OK || nothing) return rc;
  return pa::launch_prefill_mod(a, info, static_cast<cudaStream_t>(stream));
}

size_t pa_decode_shared_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                       int head_dim) {
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || !pa::head_dim_supported(head_dim))
    return 0;
  pa::DeviceInfo info;
  if (!pa::current_device_info(&info)) return 0;
  pa::DecodeSharedArgs a{};
  a.num_seqs = num_seqs > 0 ? num_seqs : 1;
  a.num_heads = num_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.grid_ctas = pa::shared_ctas(info, num_kv_heads / pa::decode_head_slab(num_kv_heads));
  return pa::shared_bind_workspace(&a, nullptr);
}

int pa_decode_shared(void* out, const void* q, const void* k_cache, const void* v_cache,
                     const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* context_lens, const int32_t* group_starts,
                     const int32_t* prefix_lens, int num_seqs, int num_groups, int num_heads,
                     int num_kv_heads, int head_dim, int dtype, int block_size,
                     int64_t num_blocks, float scale, void* workspace, size_t workspace_bytes,
                     int* dev_err, void* stream) {
  pa::DecodeSharedArgs a;
  pa::DeviceInfo info;
  bool nothing = false;
  if (num_seqs > 0 && (num_groups < 1 || num_groups > num_seqs)) return PA_ERR_SHAPE;
  if (num_seqs > pa::kMaxSharedSeqs) return PA_ERR_UNSUPPORTED;
  if (num_seqs > 0 && (!group_starts || !prefix_lens)) return PA_ERR_NULL;
  const int rc = pa::decode_prepare(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                    context_lens, num_seqs, num_heads, num_kv_heads, head_dim,
                                    dtype, block_size, num_blocks, scale, 0, dev_err, nullptr,
                                    &a, &info, &nothing);
  if (rc != PA_OK || nothing) return rc;
  a.sh.group_starts = group_starts;
  a.sh.prefix_lens = prefix_lens;
  a.sh.num_groups = num_groups;
  a.sh.boxes = pa::prefix_box_rows(block_size) > 0;
  a.grid_ctas = pa::shared_ctas(info, num_kv_heads / pa::decode_head_slab(num_kv_heads));
  const size_t need = pa::shared_bind_workspace(&a, static_cast<unsigned char*>(workspace));
  if (!workspace || workspace_bytes < need) return PA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return PA_ERR_ALIGN;
  return pa::launch_decode_shared(a, info, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace pa {

static bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1) == 0; }
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

static int check_q8_cache(const pa_q8_cache* c) {
  if (!c) return PA_ERR_NULL;
  if (c->format != PA_Q8_E4M3 && c->format != PA_Q8_INT8) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}
static int check_q8_pointers(const pa_q8_cache* c) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return PA_ERR_NULL;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
    return PA_ERR_ALIGN;
  return PA_OK;
}

// Sizes of the paged cache that a call writes or reads by slot or block.
static int check_cache_shape(int num_kv_heads, int head_dim, int block_size, int64_t num_blocks) {
  if (num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0) return PA_ERR_SHAPE;
  if (!head_dim_supported(head_dim)) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

static int check_rotary(const pa_rotary* r, int head_dim) {
  if (!r) return PA_ERR_NULL;
  if (r->rotary_dim < 16 || r->rotary_dim > head_dim || r->rotary_dim % 16 || r->num_axes < 1 ||
      r->num_axes > 16 || !isfinite(r->amplitude))
    return PA_ERR_SHAPE;
  return PA_OK;
}

// The new tokens' rows: k and v, and with rotary q too.
struct RowTensors {
  void* q_out;
  const void *q, *k, *v;
  int64_t q_out_stride, q_stride, k_stride, v_stride;
  int dtype;
  const int32_t* positions;
  int64_t pos_stride;
  const pa_rotary* rotary;  // null: keys and values only
  int num_heads;
};

// pa_store_kvcache_q8, pa_rotary_store (k_cache, v_cache) and pa_rotary_store_q8 (q8).
static int rows_entry(const RowTensors& t, void* k_cache, void* v_cache, const pa_q8_cache* q8,
                      bool to_q8, const int32_t* slot_mapping, int num_tokens, int num_kv_heads,
                      int head_dim, int block_size, int64_t num_blocks, int* dev_err,
                      void* stream, bool rotary) {
  int rc = check_cache_shape(num_kv_heads, head_dim, block_size, num_blocks);
  if (rc != PA_OK) return rc;
  if (num_tokens < 0 || (rotary && t.num_heads <= 0)) return PA_ERR_SHAPE;
  if (t.dtype != PA_DTYPE_BF16 && t.dtype != PA_DTYPE_F16) return PA_ERR_UNSUPPORTED;
  if (to_q8 && (rc = check_q8_cache(q8)) != PA_OK) return rc;
  if (rotary && (rc = check_rotary(t.rotary, head_dim)) != PA_OK) return rc;
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  const int64_t q_row = (int64_t)t.num_heads * head_dim;
  if (t.k_stride < row || t.v_stride < row) return PA_ERR_SHAPE;
  if (rotary && (t.q_stride < q_row || t.q_out_stride < q_row)) return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (!t.k || !t.v || !slot_mapping) return PA_ERR_NULL;
  if (rotary && (!t.q || !t.q_out || !t.positions || !t.rotary->turns || !t.rotary->axes))
    return PA_ERR_NULL;
  if (to_q8) {
    if ((rc = check_q8_pointers(q8)) != PA_OK) return rc;
  } else {
    if (!k_cache || !v_cache) return PA_ERR_NULL;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_ALIGN;
  }
  if (!aligned2(t.k) || !aligned2(t.v) || !aligned4(slot_mapping)) return PA_ERR_ALIGN;
  if (rotary && (!aligned2(t.q) || !aligned2(t.q_out) || !aligned4(t.positions) ||
                 !aligned4(t.rotary->axes) ||
                 (reinterpret_cast<uintptr_t>(t.rotary->turns) & 7)))
    return PA_ERR_ALIGN;
  DeviceInfo info;
  if (!current_device_info(&info)) return PA_ERR_CUDA;
  RowsArgs a{};
  a.k = t.k;
  a.v = t.v;
  a.k_stride = t.k_stride;
  a.v_stride = t.v_stride;
  bool vec = aligned16(t.k) && aligned16(t.v) && t.k_stride % 8 == 0 && t.v_stride % 8 == 0;
  if (rotary) {
    a.q_out = t.q_out;
    a.q = t.q;
    a.q_out_stride = t.q_out_stride;
    a.q_stride = t.q_stride;
    a.positions = t.positions;
    a.pos_stride = t.pos_stride;
    a.rot = *t.rotary;
    a.num_heads = t.num_heads;
    vec = vec && aligned16(t.q) && aligned16(t.q_out) && t.q_stride % 8 == 0 &&
          t.q_out_stride % 8 == 0;
  }
  a.k_cache = to_q8 ? q8->k : k_cache;
  a.v_cache = to_q8 ? q8->v : v_cache;
  a.k_scale = to_q8 ? q8->k_scale : nullptr;
  a.v_scale = to_q8 ? q8->v_scale : nullptr;
  a.slots = slot_mapping;
  a.num_tokens = num_tokens;
  a.num_kv_heads = num_kv_heads;
  a.block_size = block_size;
  a.num_slots = num_blocks * (int64_t)block_size;
  a.dev_err = dev_err;
  a.vec = vec;
  const int fmt = to_q8 ? q8->format : 0;
  const bool f16 = t.dtype == PA_DTYPE_F16;
  return rotary
             ? launch_rotary_rows(a, fmt, head_dim, f16, info, static_cast<cudaStream_t>(stream))
             : launch_store_rows(a, fmt, head_dim, f16, info, static_cast<cudaStream_t>(stream));
}

}  // namespace pa

extern "C" {

int pa_store_kvcache_q8(const void* k, const void* v, int64_t k_tok_stride, int64_t v_tok_stride,
                        int dtype, const pa_q8_cache* cache, const int32_t* slot_mapping,
                        int num_tokens, int num_kv_heads, int head_dim, int block_size,
                        int64_t num_blocks, int* dev_err, void* stream) {
  pa::RowTensors t{};
  t.k = k;
  t.v = v;
  t.k_stride = k_tok_stride;
  t.v_stride = v_tok_stride;
  t.dtype = dtype;
  return pa::rows_entry(t, nullptr, nullptr, cache, true, slot_mapping, num_tokens, num_kv_heads,
                        head_dim, block_size, num_blocks, dev_err, stream, false);
}

int pa_rotary_store(void* q_out, const void* q, const void* k, const void* v,
                    int64_t q_out_tok_stride, int64_t q_tok_stride, int64_t k_tok_stride,
                    int64_t v_tok_stride, int dtype, const int32_t* positions,
                    int64_t pos_axis_stride, const pa_rotary* rotary, void* k_cache,
                    void* v_cache, const int32_t* slot_mapping, int num_tokens, int num_heads,
                    int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                    int* dev_err, void* stream) {
  const pa::RowTensors t{q_out,        q,            k,     v,         q_out_tok_stride,
                         q_tok_stride, k_tok_stride, v_tok_stride,
                         dtype,        positions,    pos_axis_stride,  rotary, num_heads};
  return pa::rows_entry(t, k_cache, v_cache, nullptr, false, slot_mapping, num_tokens,
                        num_kv_heads, head_dim, block_size, num_blocks, dev_err, stream, true);
}

int pa_rotary_store_q8(void* q_out, const void* q, const void* k, const void* v,
                       int64_t q_out_tok_stride, int64_t q_tok_stride, int64_t k_tok_stride,
                       int64_t v_tok_stride, int dtype, const int32_t* positions,
                       int64_t pos_axis_stride, const pa_rotary* rotary,
                       const pa_q8_cache* cache, const int32_t* slot_mapping, int num_tokens,
                       int num_heads, int num_kv_heads, int head_dim, int block_size,
                       int64_t num_blocks, int* dev_err, void* stream) {
  const pa::RowTensors t{q_out,        q,            k,     v,         q_out_tok_stride,
                         q_tok_stride, k_tok_stride, v_tok_stride,
                         dtype,        positions,    pos_axis_stride,  rotary, num_heads};
  return pa::rows_entry(t, nullptr, nullptr, cache, true, slot_mapping, num_tokens, num_kv_heads,
                        head_dim, block_size, num_blocks, dev_err, stream, true);
}

uint64_t pa_rotary_turns(double inv_freq) {
  // 1 / (2 pi) in 192 binary places, most significant word first
  constexpr uint64_t kInv2Pi[3] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull,
                                   0x36d8a5664f10e410ull};
  if (!isfinite(inv_freq) || fabs(inv_freq) > 0x1p40) return 0;
  int x = 0;
  const uint64_t m = (uint64_t)ldexp(frexp(fabs(inv_freq), &x), 53);  // |inv_freq| = m 2^(x-53)
  // m / (2 pi) with 192 places, least significant word first
  uint64_t p[4];
  unsigned __int128 carry = 0;
  for (int i = 0; i < 3; ++i) {
    carry += (unsigned __int128)m * kInv2Pi[2 - i];
    p[i] = (uint64_t)carry;
    carry >>= 64;
  }
  p[3] = (uint64_t)carry;
  // times 2^(x-53), 64 places kept: shift right by 192 - 64 - (x - 53), at least 140
  const int shift = 181 - x;
  if (shift >= 256) return 0;
  auto bit = [&](int i) { return i < 256 ? p[i >> 6] >> (i & 63) & 1 : 0; };
  uint64_t r = bit(shift - 1);  // rounds
  for (int i = 0; i < 64; ++i) r += bit(shift + i) << i;
  return inv_freq < 0 ? 0 - r : r;
}

int pa_load_kvcache_q8(void* k_out, void* v_out, int dtype, const pa_q8_cache* cache,
                       const int32_t* blocks, int num_listed, int num_kv_heads, int head_dim,
                       int block_size, int64_t num_blocks, int* dev_err, void* stream) {
  int rc = pa::check_cache_shape(num_kv_heads, head_dim, block_size, num_blocks);
  if (rc != PA_OK) return rc;
  if (num_listed < 0) return PA_ERR_SHAPE;
  if (dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_F16) return PA_ERR_UNSUPPORTED;
  if ((rc = pa::check_q8_cache(cache)) != PA_OK) return rc;
  if ((int64_t)block_size * num_kv_heads > INT32_MAX / 2) return PA_ERR_UNSUPPORTED;
  if (num_listed == 0) return PA_OK;
  if (!k_out || !v_out || !blocks) return PA_ERR_NULL;
  if ((rc = pa::check_q8_pointers(cache)) != PA_OK) return rc;
  if (!pa::aligned16(k_out) || !pa::aligned16(v_out) || !pa::aligned4(blocks)) return PA_ERR_ALIGN;
  pa::DeviceInfo info;
  if (!pa::current_device_info(&info)) return PA_ERR_CUDA;
  const pa::LoadQ8Args a{k_out,          v_out,  cache->k,   cache->v,     cache->k_scale,
                         cache->v_scale, blocks, num_listed, num_kv_heads, block_size,
                         num_blocks,     dev_err};
  return pa::launch_load_q8(a, cache->format, head_dim, dtype == PA_DTYPE_F16, info,
                            static_cast<cudaStream_t>(stream));
}

int pa_decode_q8(void* out, const void* q, const pa_q8_cache* cache, const int32_t* block_tables,
                 int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                 int num_heads, int num_kv_heads, int head_dim, int dtype, int block_size,
                 int64_t num_blocks, float scale, int grid_ctas, void* workspace,
                 size_t workspace_bytes, int* dev_err, void* stream) {
  int rc = pa::check_q8_cache(cache);
  if (rc != PA_OK) return rc;
  pa::DecodeQ8Args a;
  pa::DeviceInfo info;
  bool nothing = false;
  if (num_seqs > 0 && (rc = pa::check_q8_pointers(cache)) != PA_OK) return rc;
  rc = pa::decode_prepare(out, q, cache->k, cache->v, block_tables, max_blocks_per_seq,
                          context_lens, num_seqs, num_heads, num_kv_heads, head_dim, dtype,
                          block_size, num_blocks, scale, grid_ctas, dev_err, nullptr, &a, &info,
                          &nothing);
  if (rc != PA_OK || nothing) return rc;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.auto_grid = grid_ctas == 0;
  rc = pa::decode_check_workspace(&a, info, workspace, workspace_bytes);
  if (rc != PA_OK) return rc;
  return pa::launch_decode_q8(a, cache->format, info, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
