// pa_launch.h — internal host-side launchers behind the C ABI (not exported).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pa.h"

namespace pa {

// The head dims the kernels are built for.
constexpr int kHeadDimApi = 128;
inline bool head_dim_supported(int d) { return d == 64 || d == 128; }

struct DeviceInfo {
  int device;
  int num_sms;
  int max_smem_optin;
  int cc_major;
  int cc_minor;
};

// Cached per-device properties of the current device; returns false on a CUDA error.
bool current_device_info(DeviceInfo* info);

int launch_store_kvcache(const void* k, const void* v, int64_t k_tok_stride,
                         int64_t v_tok_stride, void* k_cache, void* v_cache,
                         const int32_t* slot_mapping, int num_tokens, int num_kv_heads,
                         int head_dim, int64_t num_slots, int* dev_err, cudaStream_t stream,
                         int num_sms);

int launch_staged_write(void* base, int64_t num_rows, int64_t num_cols, int64_t row_stride,
                        int elem_bytes, const int32_t* rows, const int32_t* starts,
                        const int32_t* offsets, const void* values, int num_writes,
                        int64_t num_values, int* dev_err, cudaStream_t stream, int num_sms);

int launch_staged_upload_apply(void* base, int64_t num_rows, int64_t num_cols,
                               int64_t row_stride, int elem_bytes, const void* packed_host,
                               void* packed_dev, const pa_staged_layout* lay, int* dev_err,
                               cudaStream_t stream, int num_sms);

size_t sample_workspace_bytes(int num_rows);
int launch_gumbel_sample(int64_t* out, const void* logits, int64_t row_stride, int is_bf16,
                         int num_rows, int vocab, const float* temperatures,
                         const uint64_t* seeds, const uint64_t* offsets, void* workspace,
                         int* dev_err, cudaStream_t stream, int num_sms);

struct DecodeArgs {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int max_blocks;
  int num_seqs;
  int num_heads;
  int num_kv_heads;
  int block_size;
  int64_t num_blocks;
  float scale_log2;  // softmax scale * log2(e)
  int grid_ctas;     // CTAs along the key stream (per head slab)
  int min_tiles;     // fewest key tiles per CTA (1: every CTA of grid_ctas may take work)
  int head_dim;      // 64 or 128
  int f16;           // element type of q, caches, out: 0 = bf16, 1 = IEEE fp16
  int* counters;     // [num_seqs * num_kv_heads]
  // fused store (pa_decode_step only; null / 0 otherwise): token b's rows, its slot
  const void* k_new;
  const void* v_new;
  int64_t k_new_stride;  // elements between tokens
  int64_t v_new_stride;
  const int32_t* slot_mapping;
  float* part_o;     // [max_ctas * 2 * num_heads * head_dim]
  float* part_lse;   // [max_ctas * 2 * num_heads]
  int* dev_err;
};

// Modified scores (pa_score_mod with the factors folded to log2 units): for a query at
// absolute position p, key t scores
//   x = cap2 * tanh(q.k * cap_in) - slope_h * log2(e) * |p - t|   (cap2 > 0)
//   x = q.k * scale_log2 - slope_h * log2(e) * |p - t|            (cap2 = 0)
// and is visible when (t <= p or the call is not causal or t < prefix) and (window = 0 or
// t > p - window or t < max(sink, prefix)).
// tanh(u) = u P(u^2) for |u| < 1: P of degree 5 fitted on Chebyshev nodes of [0, 1],
// reweighted toward the largest relative error: 6e-7 relative.
constexpr float kTanhPoly[6] = {0.9999994039535522f,   -0.3332904279232025f,
                                0.13281433284282684f,  -0.051605675369501114f,
                                0.016743116080760956f, -0.0030670606065541506f};
// The same of degree 3 for |u| < 0.6: 2.2e-6 relative.
constexpr float kTanhPoly3[4] = {0.9999978542327881f, -0.33314040303230286f,
                                 0.13057856261730194f, -0.04092942550778389f};
struct ScoreModArgs {
  float cap2;                  // softcap * log2(e); 0 = no cap
  // kTanhPoly and kTanhPoly3 scaled by cap2 * cap_in^(2i+1), so that raw products go in and
  // log2 units come out; each coefficient twice, for packed arithmetic
  alignas(8) float poly[6][2];
  alignas(8) float poly3[4][2];
  float z_lim;                 // squares of raw products below which they hold: 1 / cap_in^2,
  float z_lim3;                // 0.6^2 / cap_in^2
  float cap_in;                // scale / softcap
  const float* slopes;         // [num_heads]; null = no bias
  int window;                  // 0 = none
  int sink;
  const int32_t* prefix_lens;  // [num_seqs]; null = 0
};

// pa_decode_mod: the decode with modified scores.
struct DecodeModArgs : DecodeArgs {
  ScoreModArgs mod;
};

// Where the join of pa_decode_shared finds the parts of a sequence's rows.
struct PrefixParts {  // of one KV head
  int32_t c0;   // CTA of the part that holds the unit's first step
  int32_t n;    // parts, one for each CTA from c0 on; 0 where nothing is shared
  int32_t row;  // row of the sequence's first head among a CTA's 256
  int32_t unused;
};
struct RestSegments {
  int32_t c0;  // CTA of the segment that holds the sequence's first tile
  int32_t n;   // segments, one for each CTA from c0 on; -1: the row is written already
};

// CTAs of pa_decode_shared: one per SM, and room for one of the prefixes beside every KV head
// slab's.
inline int shared_ctas(const DeviceInfo& info, int slabs) {
  return info.num_sms > slabs + 1 ? info.num_sms : slabs + 1;
}

// pa_decode_shared: the groups and the partial results (normalised rows and base-2
// log-sum-exps). Of a prefix unit or a sequence's rest, the part that holds the first step or
// tile is stored by sequence, a part that another CTA carries on by that CTA (a CTA carries
// on one unit and one sequence at most, its first; DecodeArgs::part_o and part_lse hold
// those of the rests).
struct SharedArgs {
  const int32_t* group_starts;  // [num_groups + 1]
  const int32_t* prefix_lens;   // [num_groups]
  int num_groups;
  int boxes;          // 1: the block size allows the prefix part's TMA boxes
  float* first_o;     // [num_seqs * num_heads * head_dim]: prefixes
  float* first_lse;   // [num_seqs * num_heads]
  float* more_o;      // [grid_ctas * 256 * head_dim]
  float* more_lse;    // [grid_ctas * 256]
  float* rest_o;      // [num_seqs * num_heads * head_dim]: rests
  float* rest_lse;    // [num_seqs * num_heads]
  PrefixParts* prefix;  // [num_seqs * num_kv_heads]
  RestSegments* rest;   // [num_seqs]
};

// The kernels keep the group arrays in shared memory while they plan: at most this many.
constexpr int kMaxSharedSeqs = 8192;

struct DecodeSharedArgs : DecodeArgs {
  SharedArgs sh;
};

// The new tokens of pa_decode_step (null for pa_decode and pa_decode_noalloc).
struct DecodeStepInput {
  const void* k_new;
  const void* v_new;
  int64_t k_new_stride;
  int64_t v_new_stride;
  const int32_t* slot_mapping;
};

// Argument validation and packing shared by pa_decode, pa_decode_step and
// pa_decode_noalloc (every check that does not concern the workspace). On PA_OK, *a holds
// every field but the workspace pointers, *info describes the current device and the grid
// is resolved (0 = one CTA per SM); *nothing is set when there is no sequence to launch.
int decode_prepare(void* out, const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* context_lens, int num_seqs, int num_heads, int num_kv_heads,
                   int head_dim, int dtype, int block_size, int64_t num_blocks, float scale,
                   int grid_ctas, int* dev_err, const DecodeStepInput* step, DecodeArgs* a,
                   DeviceInfo* info, bool* nothing);
// Points a's counters and partial-result slots into `ws`, laid out for layout_ctas CTAs
// (decode_workspace_layout); returns the bytes that layout needs. ws may be null (only
// the size is wanted then).
size_t decode_bind_workspace(DecodeArgs* a, unsigned char* ws, int layout_ctas);

// With the automatic grid, a CTA takes at least this many key tiles (64 KB of K and V
// each at H_kv = 8): a short stream is then cut into fewer, longer CTA ranges, so that a
// small batch's sequences are split into fewer segments to combine.
constexpr int kDecodeMinTilesPerCta = 4;

// Maximum CTAs along the key stream that a decode workspace is sized for.
int decode_max_ctas(const DeviceInfo& info);
// Workspace layout: byte offsets of the counters, partial LSEs and partial outputs.
void decode_workspace_layout(int num_seqs, int num_heads, int num_kv_heads, int max_ctas,
                             size_t* off_counters, size_t* off_lse, size_t* off_o,
                             size_t* total);
// Tokens per TMA box of the prefix part: the largest power of two that divides the block
// size, at most a tile; 0 below the 8 rows of a swizzle atom.
inline int prefix_box_rows(int block_size) {
  const int tb = block_size & -block_size;
  return tb > 128 ? 128 : (tb < 8 ? 0 : tb);
}
// Head slab (KV heads handled by one CTA) for a given num_kv_heads: 8, 4, 2 or 1.
int decode_head_slab(int num_kv_heads);
bool decode_supported(int num_heads, int num_kv_heads);
int launch_decode(const DecodeArgs& a, const DeviceInfo& info, cudaStream_t stream);
// The CUDA-core decode (and fused-step) instantiations with fp16 elements, in their own
// translation units.
int launch_decode_d128_f16(const DecodeArgs& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_step_d128_f16(const DecodeArgs& a, const DeviceInfo& info, cudaStream_t stream);
// The tensor-core path (decode_tc.cuh).
int launch_decode_tc(const DecodeArgs& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_step_tc(const DecodeArgs& a, const DeviceInfo& info, cudaStream_t stream);
// Modified scores: the tensor-core kernel, every shape.
int launch_decode_mod(const DecodeModArgs& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_mod_d64(const DecodeModArgs& a, const DeviceInfo& info, cudaStream_t stream);
// pa_decode_shared: one launch over the keys (shared_decode.cuh), one translation unit for each
// head_dim and element type, then the join of the parts (shared_join.cu).
int launch_decode_shared(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream);
int launch_shared_d64_bf16(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream);
int launch_shared_d64_f16(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream);
int launch_shared_d128_bf16(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream);
int launch_shared_d128_f16(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream);
// Shapes that take the tensor-core path: every group of 3..8 query heads per KV head, and
// groups of 1 or 2 unless the head dimension is 128 and one slab holds all KV heads
// (num_kv_heads 1, 2, 4 or 8), the case where a CUDA-core tile is one contiguous run of
// cache rows. Elsewhere the tensor-core kernel's TMA boxes stream faster.
inline bool decode_uses_tc(int num_heads, int num_kv_heads, int head_dim) {
  const int g = num_heads / num_kv_heads;
  if (g >= 3) return true;
  const bool one_slab = num_kv_heads == 1 || num_kv_heads == 2 || num_kv_heads == 4 ||
                        num_kv_heads == 8;
  return !(head_dim == 128 && one_slab);
}
// The same kernel with the store of token b (k_new/v_new row b) at slot_mapping[b] fused in;
// the caches are written, so a.k_cache / a.v_cache must point to writable memory.
int launch_decode_step(const DecodeArgs& a, const DeviceInfo& info, cudaStream_t stream);

struct PrefillArgs {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* cu_seqlens_q;
  const int32_t* cu_seqlens_k;
  int max_blocks;
  int num_seqs;
  int max_seqlen_q;
  int max_seqlen_k;
  int num_heads;
  int num_kv_heads;
  int block_size;
  int64_t num_blocks;
  int causal;
  float scale_log2;
  int head_dim;  // 64 or 128
  int f16;       // element type of q, caches, out: 0 = bf16, 1 = IEEE fp16
  int* dev_err;
  int persistent;  // set by the launcher: 1 = one CTA per SM walking a sorted unit list
};

// pa_prefill_mod: the prefill with modified scores.
struct PrefillModArgs : PrefillArgs {
  ScoreModArgs mod;
};

bool prefill_supported(int num_heads, int num_kv_heads, int block_size);
int launch_prefill(const PrefillArgs& a, const DeviceInfo& info, cudaStream_t stream);
int launch_prefill_mod(const PrefillModArgs& a, const DeviceInfo& info, cudaStream_t stream);
// One translation unit for each head_dim, element type and form (prefill_kernel.cuh).
template <int D, bool F16, int FORM>
int launch_prefill_form(const PrefillModArgs& a, const DeviceInfo& info, cudaStream_t stream,
                        const CUtensorMap& mk, const CUtensorMap& mv);
// The prefill instantiations other than head_dim 128 with bf16, one translation unit each.
int launch_prefill_d64_bf16(const PrefillArgs& a, const DeviceInfo& info, cudaStream_t stream,
                            const CUtensorMap& mk, const CUtensorMap& mv);
int launch_prefill_d64_f16(const PrefillArgs& a, const DeviceInfo& info, cudaStream_t stream,
                           const CUtensorMap& mk, const CUtensorMap& mv);
int launch_prefill_d128_f16(const PrefillArgs& a, const DeviceInfo& info, cudaStream_t stream,
                            const CUtensorMap& mk, const CUtensorMap& mv);

}  // namespace pa
