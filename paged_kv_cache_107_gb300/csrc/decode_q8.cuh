// decode_q8.cuh — paged decode attention over an 8-bit cache (pa_q8_cache) on the tensor cores:
// warp-level mma.sync m16n8k16 with fp16 operands and fp32 accumulators.
//
// With codes kc, vc and scales ks, vs of key t, query row q and c = softmax scale * log2 e:
//   x_t = c ks_t (q . kc_t),  m = max x,  l = sum 2^(x_t - m),  o = sum (2^(x_t - m) vs_t) vc_t / l
// The work split (stream-K over key tiles), the partial results and their order are those of
// decode_kernel.cuh and decode_tc.cuh. Bound by the bytes of codes and scales: 256 sequences of
// 100 to 2,048 positions (16 / 8 heads of 128) take 85 us, 6.7 TB/s or 0.98 of the copy rate; 8 of
// 32k to 131k with 32 / 8 heads 217, 7.0 TB/s; 200 of up to 4,096 with 32 / 8 fp16 heads of 64 (int8)
// 69 us at block size 32 and more (6.0 TB/s) and 76 at 16, whose 8 KB runs the memory serves more
// slowly. Without any products these take 83.6, 218, 63 and 67. With few KV heads the rows are short
// (256 sequences, two queries a KV head: 28 us at 1, 37 at 2, 55 at 3, 51 at 4 KV heads, of which the
// bytes are 10, 21, 31 and 42). Block sizes that no power of two from 8 up divides are copied by one
// warp a token at a time: 763 us at 4, 748 at 20, 745 at 100, 824 at 1 for the 256 sequences, 86 at 16.
// What differs from the 16-bit kernels:
//
//  * A code is half as many bytes, so a stage of 64 KB holds twice the tokens, and every byte has
//    to be widened: e4m3 by the hardware's conversion to fp16 (exact), int8 by placing the byte
//    in an fp16 number (q8.cuh). Nothing is widened in shared memory: a register of four codes
//    becomes two fp16 words of an MMA operand. (int8 keys x could enter the scores as the 1152 + x
//    that they come as, with sums that start at -1152 sum q: 72.2 us instead of 75.5 for the 200
//    sequences. But the fp32 sums would pass through 2,431 sum |q|, where each of the D / 16
//    MMAs rounds: scores of queries far from zero mean lose more than an fp16 result's own rounding.)
//  * Both products are taken transposed, S^T = K Q^T and O^T = V^T W^T: 16 tokens, or 16 dims, are
//    the 16 rows of an MMA and the up to 8 heads of a group its 8 columns, so that no row is
//    padding (with the heads as rows half of them are: 114 us against 89 for the 256 sequences).
//    K: ldmatrix gives a lane four consecutive dims of a token; its two words stand for dims 4i,
//    4i+1 and 4i+2, 4i+3, and the queries are loaded in the same order.
//    V: the transposing ldmatrix moves 16-bit pieces, so a register holds dims 2i, 2i+1 of two
//    tokens. Its even bytes are a word of row i, its odd bytes of row i + 8: row r of a chunk
//    of 16 dims is dim 2 (r mod 8) + r / 8.
//    W: a warp's weights (token by head) become the second product's operand (head by token)
//    with movmatrix.
//  * A warp takes 32 tokens of a stage (64 with heads of 64), a lane two heads' scores of four
//    (eight) of them. The running maximum is moved only when one of these scores exceeds it (one
//    vote): most tiles need no shuffle and no rescaling.
//  * The K scale multiplies the score. The V scale is taken into the weight, which then enters the
//    product as the sum of two fp16 numbers: w_t = p_t vs_t 2^(14-E), E the exponent of the largest
//    vs met so far by the warp (when it grows the accumulators are rescaled), so that w < 2^15 and
//    what is rounded off lies 2^-39 below the largest scale or 2^-22 below w itself. With one
//    fp16 number, 2^-11, an fp16 result's error grows by half (0.00030 of its size against 0.00021),
//    and bf16 results come out a unit of the last place away from the exact one's rounding wherever
//    that lies near a tie. The second product costs 0 to 4 %: with bf16 results 84.6 -> 84.8 us for
//    the 256 sequences, 70.1 -> 72.5 for the 200, 54.6 -> 56.9 for 256 with 32 / 4 heads of 128.
//  * bf16 queries go to fp16 with a power of two for each head (row_to_f16 below).
//  * Rows of shared memory are 128 bytes with the 128-byte swizzle: a head of 128 dims, or two
//    heads of 64, which lie side by side in the cache (half as many rows for the copies: 76.0 us for the
//    200 sequences at block size 16, with rows of one head 77.5). A single head of 64 has 64-byte rows
//    and the 64-byte swizzle.
//  * Stages of 64 KB, as elsewhere: with half as many tokens of 64 dims in each the same 200
//    sequences take 82.5 us (92.6 at block size 16).
//  * Scales come beside the codes, [head][token] of each box, by TMA; their slots are padded to
//    128 bytes (a TMA destination's alignment). Fetched by the producer's lanes instead, 16 bytes
//    at a time, the same batches take 2 to 4 % longer.
#pragma once

#include "decode_tc.cuh"
#include "q8.cuh"

namespace pa {
namespace {

template <int HS, int D>
struct Q8Cfg {
  static constexpr int SUB = D == 64 ? 2 : 1;       // a warp takes 32 * SUB tokens of a stage
  static constexpr int T = 256 * SUB / HS;          // tokens per stage
  static constexpr int WPH = kConsumerWarps / HS;   // warps per KV head (token split)
  static constexpr int KV_BYTES = HS * T * D;
  static constexpr int HPR = D == 64 && HS > 1 ? 2 : 1;  // heads of one shared-memory row
  static constexpr int ROW = HPR * D;               // 128 bytes, or 64 for a single head of 64
  static constexpr int SC_BYTES = T * (4 * HS > 16 ? 4 * HS : 16);  // boxes of 8 tokens, padded
  static constexpr int STAGE_BYTES = (2 * (KV_BYTES + SC_BYTES) + 1023) / 1024 * 1024;
  static constexpr int Q_BYTES = HS * kTcGMax * D * 2;
  static constexpr int CTRL_BYTES = 1024;
  static constexpr int BUDGET = 227 * 1024 - 1024 - CTRL_BYTES;  // less the alignment slack
  static constexpr int QS = (3 * STAGE_BYTES + 2 * Q_BYTES <= BUDGET) ? 2 : 1;
  static constexpr int STAGES = (BUDGET - QS * Q_BYTES) / STAGE_BYTES;
  static constexpr int MERGE_FLOATS = kTcGMax * (D + 2);
  static constexpr size_t SMEM =
      1024 + (size_t)STAGES * STAGE_BYTES + (size_t)QS * Q_BYTES + CTRL_BYTES;
  static_assert(STAGES >= 2, "at least two stages");
  static_assert(sizeof(TcCtrl<STAGES>) <= CTRL_BYTES, "control block");
  static_assert(HS * (WPH - 1) * MERGE_FLOATS * 4 <= 2 * KV_BYTES, "merge scratch");
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// D (16x8) += A (16x16) B (16x8), fp16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8x8 matrix of 16-bit elements held by the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The last arrival for (sequence, KV head): joins the partials of its nseg CTAs c_lo.. in CTA order
// and writes the G rows from head hg0 on. One warp; lane s holds the weights of segment s of a
// chunk of 32. The partial rows of two heads and 8 segments (16 of 64 dims) are asked for together, beside the
// log-sum-exps that will weigh them, so that up to as many segments cost one round trip to memory
// for each pair of heads. (combine_partials of decode_kernel.cuh takes one for each segment here,
// within the registers that its kernel leaves it: 8 segments cost 5 us. Out of line, this one has
// the registers to itself.)
template <int D, bool F16>
__device__ __noinline__ void combine_q8(const float* part_o, const float* part_lse, uint16_t* out,
                                        int H, int hg0, int G, int c_lo, int nseg,
                                        bool first_slot, int lane) {
  constexpr int CPL = D / 32, SU = 32 / CPL;
#pragma unroll 1
  for (int h0 = 0; h0 < G; h0 += 2) {
    const int two = h0 + 1 < G ? 1 : 0;  // 0: the second of the pair repeats the first
    // row of a segment's partials: a CTA's slot 1 where the sequence is not its first
    auto row = [&](int seg, int q) {
      return ((int64_t)(c_lo + seg) * 2 + (seg == 0 && first_slot ? 1 : 0)) * H + hg0 + h0 + q * two;
    };
    float po[SU][2][CPL];
    auto ask = [&](int s0) {  // (past the last segment: the last one again, with no weight)
#pragma unroll
      for (int u = 0; u < SU; ++u)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float* src = part_o + row(min(s0 + u, nseg - 1), q) * D + lane * CPL;
          if constexpr (CPL == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
            po[u][q][0] = v.x, po[u][q][1] = v.y, po[u][q][2] = v.z, po[u][q][3] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
            po[u][q][0] = v.x, po[u][q][1] = v.y;
          }
        }
    };
    float acc[2][CPL], m_h[2], den[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      m_h[q] = -INFINITY;
      den[q] = 0.f;
#pragma unroll
      for (int e = 0; e < CPL; ++e) acc[q][e] = 0.f;
    }
#pragma unroll 1
    for (int s0 = 0; s0 < nseg; s0 += 32) {
      const int nb = min(32, nseg - s0);
      float w[2];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        w[q] = lane < nb ? __ldcg(part_lse + row(s0 + lane, q)) : -INFINITY;
      ask(s0);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float bm = w[q];
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, m));
        const float nm = fmaxf(m_h[q], bm);
        const float al = m_h[q] == nm ? 1.f : fast_exp2(m_h[q] - nm);
        m_h[q] = nm;
        // (a segment without keys weighs nothing; a NaN stays one)
        w[q] = w[q] == -INFINITY ? 0.f : fast_exp2(w[q] - nm);
        float sum = w[q];
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        den[q] = den[q] * al + sum;
#pragma unroll
        for (int e = 0; e < CPL; ++e) acc[q][e] *= al;
      }
#pragma unroll 1
      for (int j0 = 0; j0 < nb; j0 += SU) {
        if (j0 > 0) ask(s0 + j0);
#pragma unroll
        for (int u = 0; u < SU; ++u)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float wj = __shfl_sync(0xffffffffu, w[q], (j0 + u) & 31);
            if (j0 + u < nb) {
#pragma unroll
              for (int e = 0; e < CPL; ++e) acc[q][e] = fmaf(wj, po[u][q][e], acc[q][e]);
            }
          }
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (q == 1 && !two) break;
      const float inv = den[q] == 0.f ? 0.f : 1.f / den[q];
      uint16_t* dst = out + (int64_t)(h0 + q) * D + lane * CPL;
      if constexpr (CPL == 4) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(f2_elt2<F16>(acc[q][0] * inv, acc[q][1] * inv),
                                                    f2_elt2<F16>(acc[q][2] * inv, acc[q][3] * inv));
      } else {
        *reinterpret_cast<uint32_t*>(dst) = f2_elt2<F16>(acc[q][0] * inv, acc[q][1] * inv);
      }
    }
  }
}

// One 3-D TMA box into shared memory.
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, int c0, int c1,
                                                 int c2, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)),
      "l"(policy)
      : "memory");
}
// The same boxes into L2 only.
__device__ __forceinline__ void prefetch_box_4d(const CUtensorMap* map, int c0, int c1, int c2,
                                                int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ void prefetch_box_3d(const CUtensorMap* map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}

struct Q8Maps {
  CUtensorMap k, v, ks, vs;
};

// A lane's part of a query, dims 16c + 4 tig .. + 3 of every chunk c, as fp16. bf16 queries are
// scaled by 2^(14-e), e the exponent of the query's largest magnitude (at least -112): exact but
// for elements 2^28 and more below that largest. The query sits in the four lanes of a quad.
// Returns the factor that undoes it.
template <int KC>
__device__ __forceinline__ float row_to_f16(uint32_t (&qa)[KC][2]) {
  uint32_t top = 0u;
#pragma unroll
  for (int c = 0; c < KC; ++c)
    top = __vmaxu2(top, __vmaxu2(qa[c][0] & 0x7fff7fffu, qa[c][1] & 0x7fff7fffu));
  top = max(top & 0xffffu, top >> 16);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int e = max((int)(top >> 7) - 127, -112);
  const float up = pow2f(14 - e);
#pragma unroll
  for (int c = 0; c < KC; ++c)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float lo, hi;
      bf16x2_to_f32(qa[c][i], lo, hi);
      qa[c][i] = f2_elt2<true>(lo * up, hi * up);
    }
  return pow2f(e - 14);
}

template <int HS, int D, int FMT, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_q8_kernel(const __grid_constant__ Q8Maps tm, const DecodeQ8Args a, const int tb) {
  using C = Q8Cfg<HS, D>;
  using Ctl = TcCtrl<C::STAGES>;
  constexpr int S = C::STAGES, T = C::T;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* qbuf = smem + (size_t)S * C::STAGE_BYTES;
  Ctl& ctl = *reinterpret_cast<Ctl*>(qbuf + (size_t)C::QS * C::Q_BYTES);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int c = (int)blockIdx.x, slab = (int)blockIdx.y, nctas = (int)gridDim.x;
  const int H = a.num_heads;
  const int Hk = a.num_kv_heads;
  const int G = H / Hk;  // 1..8
  const int cap = a.max_blocks * a.block_size;
  const int B = a.num_seqs;
  // (unsigned: a context may end near 2^31)
  auto tiles_in = [](int n) { return (int)(((unsigned)n + T - 1) / T); };
  auto tiles_of = [&](int b) { return tiles_in(load_ctx(a.context_lens, b, cap)); };

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], kConsumerWarps);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&ctl.q_full[q], 1);
      mbar_init(&ctl.q_empty[q], kConsumerWarps);
    }
    mbar_init(&ctl.seg_bar, kConsumerWarps);
    if (C::WPH > 1)
      for (int j = 0; j < HS; ++j) mbar_init(&ctl.merge_bar[j], C::WPH - 1);
    ctl.found = 0;
    ctl.abort = 0;
    ctl.b0 = 0;
    ctl.pb0 = 0;
    fence_mbar_init();
  }
  if (tid < S) ctl.meta[tid] = StageMeta{};  // a first wait may run out: no keys
  pdl_launch_dependents();

  // ---- prologue: total tiles, then the sequence that holds this CTA's first tile -----
  constexpr int kScan = kConsumerWarps * 32;  // sequences scanned at a time
  int64_t NT = 0, x0 = 0, x1 = 0;
  int g_eff = 0, held = 0;  // CTAs that own tiles; sequences that hold keys
  // a chunk of kScan sequences: tiles of sequence base + tid, of those before it, of all
  auto scan = [&](int base, int64_t* before, int64_t* all) {
    const int b = base + tid;
    const int n = tid < kScan && b < B ? tiles_of(b) : 0;
    held += __syncthreads_count(n > 0);
    int64_t incl = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += y;
    }
    if (lane == 31) ctl.red[warp] = incl;
    __syncthreads();
    *before = incl - n;
    *all = 0;
#pragma unroll
    for (int w = 0; w < kConsumerWarps; ++w) {
      const int64_t r = ctl.red[w];
      if (w < warp) *before += r;
      *all += r;
    }
    return n;
  };
  auto split = [&]() {  // this CTA's share of NT tiles
    int64_t want = NT;
    if (a.auto_grid) {
      // A tile takes a CTA 0.95 us, each segment of a sequence its combine 0.11 us for every pair
      // of heads of 128: with g CTAs NT / g of the one and g / held of the other, least at this g
      // (one sequence of 200, 1,000, 30,000 keys 7.5, 9.3, 26.2 us; with at least four tiles for
      // each CTA 10.6, 10.5, 28.9; of 1,000 with 8 heads a group 14.5, with a tile for each CTA
      // 18.5). Rows of 64 are joined in a quarter of the time (1,000, 30,000 keys of 32 / 8 heads
      // of 64 8.9, 25.9 us; with the ratio of 128 10.4, 29.6). Then as few CTAs as keep the longest
      // share (16 of 1,000: 12.5 us, 14.4 without).
      constexpr float kRatio = D == 128 ? 8.6f : 34.f;
      want = (int64_t)sqrtf((float)NT * (float)held * (kRatio / (float)((G + 1) / 2)));
      want = want < 1 ? 1 : want;
      if (want > nctas) want = nctas;
      if (want < NT) {
        const int64_t share = (NT + want - 1) / want;
        want = (NT + share - 1) / share;
      } else {
        want = NT;
      }
    }
    g_eff = (int)(want < (int64_t)nctas ? want : (int64_t)nctas);
    if (c < g_eff) {
      x0 = tile_begin(c, NT, g_eff);
      x1 = tile_begin(c + 1, NT, g_eff);
    }
  };
  auto holds = [&](int b, int64_t p, int n) {  // tiles p .. p + n - 1 are those of sequence b
    if (n > 0 && x0 < x1 && p <= x0 && x0 < p + n) {
      ctl.b0 = b;
      ctl.pb0 = p;
      ctl.found = 1;
    }
  };
  for (int b = tid; b < B; b += kThreads) {
    const int raw = __ldg(a.context_lens + b);
    if ((raw < 0 || raw > cap) && (b % nctas) == c && slab == 0)
      set_dev_err(a.dev_err, PA_DEV_ERR_CONTEXT);
  }
  if (B <= kScan) {
    int64_t p;
    const int n = scan(0, &p, &NT);
    split();
    holds(tid, p, n);
  } else {
    for (int base = 0; base < B; base += kScan) {
      int64_t p, all;
      scan(base, &p, &all);
      NT += all;
      __syncthreads();
    }
    split();
    int64_t running = 0;
    for (int base = 0; base < B && running <= x0; base += kScan) {
      int64_t p, all;
      const int n = scan(base, &p, &all);
      holds(base + tid, running + p, n);
      running += all;
      __syncthreads();
    }
  }
  __syncthreads();

  const bool boxes = tb > 0;
  const int nbx = boxes ? T / tb : 0;  // boxes of a full tile
  // Before the wait the producer warms L2 with what its first tiles read: the codes and the
  // block ids, which no earlier kernel of the step writes but for the new tokens' rows
  // (a line warmed too early is the one that the store then updates).
  if (warp == kProducerWarp && boxes && x0 < x1 && ctl.found) {
    int b = ctl.b0;
    int64_t pb = ctl.pb0;
    int hi = load_ctx(a.context_lens, b, cap);
    int nb = tiles_in(hi);
    for (int64_t x = x0; x < x1 && x < x0 + S; ++x) {
      while (x >= pb + nb && b + 1 < B) {
        pb += nb;
        ++b;
        hi = load_ctx(a.context_lens, b, cap);
        nb = tiles_in(hi);
      }
      const int tok0 = (int)(x - pb) * T;
      const int count = min(T, hi - tok0);
      for (int i = lane; i < nbx && i * tb < count; i += 32) {
        const int pos = tok0 + i * tb;
        const int id = __ldg(a.block_tables + (int64_t)b * a.max_blocks + pos / a.block_size);
        if (id < 0 || (int64_t)id >= a.num_blocks) continue;
        const int off = pos % a.block_size;
        prefetch_box_4d(&tm.k, 0, off, slab * (HS / C::HPR), id);
        prefetch_box_4d(&tm.v, 0, off, slab * (HS / C::HPR), id);
        prefetch_box_3d(&tm.ks, off, slab * HS, id);
        prefetch_box_3d(&tm.vs, off, slab * HS, id);
      }
    }
  }
  pdl_wait();

  {  // zero rows of empty (or invalid) sequences assigned to this CTA: one warp per row
    const int heads = HS * G;
    for (int b = c + warp * nctas; b < B; b += (kThreads / 32) * nctas) {
      if (load_ctx(a.context_lens, b, cap) != 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                            ((int64_t)b * H + slab * heads) * D);
      for (int i = lane; i < heads * D / 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
    }
  }
  if (x0 >= x1) return;
  if (!ctl.found) {  // context_lens changed under the kernel
    if (tid == 0) set_dev_err(a.dev_err, PA_DEV_ERR_CONTEXT);
    return;
  }
  // the end of a segment reads these again: nothing of the split stays in registers meanwhile
  if (tid == 0) {
    ctl.nt = NT;
    ctl.x0 = x0;
    ctl.g_eff = g_eff;
  }
  __syncthreads();
  const int64_t n_tiles = x1 - x0;
  volatile int* abort_flag = &ctl.abort;
  auto gave_up = [&]() {
    if (lane == 0) {
      ctl.abort = 1;
      set_dev_err(a.dev_err, PA_DEV_ERR_TIMEOUT);
    }
  };
  // boxes of tbl tokens, [heads of a row][token][row]; 16-byte chunk ch of token t's row sits at
  // chunk ch ^ swizzle(t)
  auto swizzle = [](int t) { return C::ROW == 128 ? t & 7 : (t >> 1) & 3; };
  const int tbl = tb > 0 ? tb : T;
  const int lg_tbl = __ffs(tbl) - 1;
  const int sc_slot = max(HS * tbl * 4, 128);

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------------ producer
    const uint64_t policy = policy_evict_first();
    if (tb > 0 && lane == 0) {
      prefetch_tensor_map(&tm.k);
      prefetch_tensor_map(&tm.v);
      prefetch_tensor_map(&tm.ks);
      prefetch_tensor_map(&tm.vs);
    }
    const int box_bytes = HS * tb * (D + 4);
    int b = ctl.b0;
    int64_t pb = ctl.pb0;
    int hi = load_ctx(a.context_lens, b, cap);
    int nb = tiles_in(hi);
    int q_n = 0;  // segments whose Q has been issued
    int s = 0;
    uint32_t phase = 0;  // of the stage's uses
    for (int64_t it = 0; it < n_tiles; ++it, s = s + 1 == S ? 0 : s + 1, phase ^= (s == 0)) {
      const int64_t x = x0 + it;
      while (x >= pb + nb && b + 1 < B) {
        pb += nb;
        ++b;
        hi = load_ctx(a.context_lens, b, cap);
        nb = tiles_in(hi);
      }
      const int lt = (int)(x - pb);
      const int tok0 = lt * T;
      const int count = min(T, hi - tok0);
      const int32_t* table = a.block_tables + (int64_t)b * a.max_blocks;
      int flags = 0;
      if (x == x0 || lt == 0) flags |= kFlagFirst;
      if (x == x1 - 1 || lt == nb - 1) flags |= kFlagLast;
      if (pb >= x0 && pb + nb <= x1) flags |= kFlagWhole;
      // this lane's boxes: tokens tok0 + i * tb .. + tb - 1 for i = lane, lane + 32, inside one
      // block each
      constexpr int kBoxes = T / 8 > 32 ? 2 : 1;
      int blk[kBoxes], off[kBoxes], nbox = 0;
#pragma unroll
      for (int r = 0; r < kBoxes; ++r) {
        const int i = lane + 32 * r;
        blk[r] = -1;
        off[r] = 0;
        if (i < nbx && i * tb < count) {
          const int pos = tok0 + i * tb;
          const int id = __ldg(table + pos / a.block_size);
          off[r] = pos % a.block_size;
          if (id >= 0 && (int64_t)id < a.num_blocks) blk[r] = id;
          else set_dev_err(a.dev_err, PA_DEV_ERR_BLOCK_ID);
        }
        nbox += __popc(__ballot_sync(0xffffffffu, blk[r] >= 0));
      }
      if (it >= S && !mbar_wait(&ctl.empty[s], phase ^ 1u, abort_flag)) gave_up();
#ifdef PA_TEST_DELAY_LAST_TILE_CYCLES
      // test build only (decode_kernel.cuh): the consumers' wait for the last tile runs out
      if (it == n_tiles - 1) {
        const long long t_hold = clock64();
        while (clock64() - t_hold < (long long)(PA_TEST_DELAY_LAST_TILE_CYCLES)) {
        }
      }
#endif
      unsigned char* st = smem + (size_t)s * C::STAGE_BYTES;
      unsigned char* st_sc = st + 2 * C::KV_BYTES;
      if (lane == 0) {
        StageMeta& m = ctl.meta[s];
        m.pb = pb;
        m.b = b;
        m.tok0 = tok0;
        m.count = count;
        m.nb = nb;
        m.flags = flags;
        if (tb > 0) mbar_arrive_expect_tx(&ctl.full[s], (uint32_t)(nbox * 2 * box_bytes));
      }
      __syncwarp();
      if (tb > 0) {
#pragma unroll
        for (int r = 0; r < kBoxes; ++r) {
          if (blk[r] < 0) continue;
          const int i = lane + 32 * r;
          tma_load_4d_hint(st + i * HS * tb * D, &tm.k, 0, off[r], slab * (HS / C::HPR), blk[r],
                           &ctl.full[s], policy);
          tma_load_3d_hint(st_sc + i * sc_slot, &tm.ks, off[r], slab * HS, blk[r], &ctl.full[s],
                           policy);
          tma_load_4d_hint(st + C::KV_BYTES + i * HS * tb * D, &tm.v, 0, off[r],
                           slab * (HS / C::HPR), blk[r], &ctl.full[s], policy);
          tma_load_3d_hint(st_sc + C::SC_BYTES + i * sc_slot, &tm.vs, off[r], slab * HS, blk[r],
                           &ctl.full[s], policy);
        }
      } else {
        // 16-byte copies into the same swizzled layout, one box of T tokens, a token at a time
        constexpr int CH = D / 16;  // 16-byte chunks of one head's row
        for (int t = 0; t < count; ++t) {
          const int pos = tok0 + t;
          const int id = __ldg(table + pos / a.block_size);
          const int in = pos % a.block_size;
          if (id < 0 || (int64_t)id >= a.num_blocks) {
            if (lane == 0) set_dev_err(a.dev_err, PA_DEV_ERR_BLOCK_ID);
            continue;
          }
          const int64_t row =
              (((int64_t)id * a.block_size + in) * Hk + slab * HS) * D;  // HS * D bytes
          for (int i = lane; i < 2 * HS * CH; i += 32) {
            const int kv = i / (HS * CH), jj = i / CH % HS, ch = i % CH;
            const unsigned char* src =
                static_cast<const unsigned char*>(kv ? a.v_cache : a.k_cache) + row + jj * D + ch * 16;
            cp_async16(st + kv * C::KV_BYTES + ((jj / C::HPR) * T + t) * C::ROW +
                           (((jj % C::HPR * CH + ch) ^ swizzle(t)) << 4),
                       src);
          }
          if (lane < 2 * HS) {
            const int kv = lane / HS, jj = lane % HS;
            const float* src = (kv ? a.v_scale : a.k_scale) +
                               ((int64_t)id * Hk + slab * HS + jj) * a.block_size + in;
            cp_async4(st_sc + kv * C::SC_BYTES + (jj * T + t) * 4, src);
          }
        }
        cp_async_arrive(&ctl.full[s]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.full[s]);
      }
      if (flags & kFlagFirst) {
        // Q of the segment (HS*G rows of D, contiguous) into its slot
        const int qs = q_n % C::QS;
        if (q_n >= C::QS &&
            !mbar_wait(&ctl.q_empty[qs], (uint32_t)(((q_n / C::QS) - 1) & 1), abort_flag))
          gave_up();
        if (lane == 0) {
          const uint32_t q_bytes = (uint32_t)(HS * G * D * 2);
          mbar_arrive_expect_tx(&ctl.q_full[qs], q_bytes);
          bulk_g2s(qbuf + (size_t)qs * C::Q_BYTES,
                   static_cast<const uint16_t*>(a.q) + ((int64_t)b * H + (int64_t)slab * HS * G) * D,
                   q_bytes, &ctl.q_full[qs]);
        }
        ++q_n;
      }
    }
    // copies still in flight land before the producer leaves
    for (int64_t it = n_tiles > S ? n_tiles - S : 0; it < n_tiles; ++it)
      mbar_wait_copies(&ctl.full[it % S], (uint32_t)((it / S) & 1));
    for (int n = q_n > C::QS ? q_n - C::QS : 0; n < q_n; ++n)
      mbar_wait_copies(&ctl.q_full[n % C::QS], (uint32_t)((n / C::QS) & 1));
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int j = warp / C::WPH;    // KV head within the slab
  const int w = warp % C::WPH;    // token group within the tile
  const int kvh = slab * HS + j;  // global KV head
  const int gid = lane >> 2, tig = lane & 3;
  constexpr int KC = D / 16;      // chunks of 16 dims
  uint32_t qa[KC][2];             // Q of head gid: dims 16 kc + 4 tig, +1 and +2, +3
  // O of heads 2 tig, 2 tig + 1: dims 16 kc + 2 gid (elements 0, 1), 16 kc + 2 gid + 1 (2, 3)
  float o[KC][4];
  // of heads 2 tig, + 1: running max (log2 units), the same but 0 while it is -inf, this lane's
  // part of the sum, c over the power of two in the fp16 queries
  float m_run[2], m_ref[2], l_part[2], cq[2];
  constexpr int kE0 = -112;
  int e_run = kE0;                // exponent of the largest value scale so far
  auto reset = [&]() {
#pragma unroll
    for (int n = 0; n < KC; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m_run[i] = -INFINITY;
      m_ref[i] = l_part[i] = 0.f;
    }
    e_run = kE0;
    cq[0] = cq[1] = 0.f;
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) qa[kc][0] = qa[kc][1] = 0u;
  };
  reset();

  // row that holds token t of head j in a code tile, and the token's scale
  auto row_off = [&](int t) -> int {
    return ((((t >> lg_tbl) * (HS / C::HPR) + j / C::HPR) << lg_tbl) + (t & (tbl - 1))) * C::ROW;
  };
  auto sc_off = [&](int t) -> int {
    return (t >> lg_tbl) * sc_slot + ((j << lg_tbl) + (t & (tbl - 1))) * 4;
  };
  // chunk 2p + hi of the head sits at chunk (ch0 + 2p + hi) ^ sw of the row, ch0 the head's first;
  // a lane's ldmatrix rows all have the same sw
  const int ch0 = (j % C::HPR) * (D / 16);
  const int sw = swizzle(lane & 7);
  const uint32_t sw_hi = (uint32_t)((sw & 6) ^ ch0) << 4;
  const int hi = lane >> 4;  // which of a pair of chunks this lane's ldmatrix row is of
  const uint32_t smem_base = smem_u32(smem);

  int seg_count = 0;
  int q_n = 0;
  int s = 0;
  uint32_t phase = 0;
  for (int64_t it = 0; it < n_tiles; ++it, s = s + 1 == S ? 0 : s + 1, phase ^= (s == 0)) {
    if (!mbar_wait(&ctl.full[s], phase, abort_flag)) gave_up();
    const StageMeta& meta = ctl.meta[s];
    const int count = meta.count, flags = meta.flags;
    unsigned char* Kst = smem + (size_t)s * C::STAGE_BYTES;
    unsigned char* Vst = Kst + C::KV_BYTES;
    const unsigned char* ksc = Kst + 2 * C::KV_BYTES;
    const unsigned char* vsc = ksc + C::SC_BYTES;

    if (flags & kFlagFirst) {
      const int qs = q_n % C::QS;
      if (!mbar_wait(&ctl.q_full[qs], (uint32_t)((q_n / C::QS) & 1), abort_flag)) gave_up();
      const unsigned char* Qst = qbuf + (size_t)qs * C::Q_BYTES;
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) {
        uint2 x = make_uint2(0u, 0u);
        if (gid < G)
          x = *reinterpret_cast<const uint2*>(Qst + ((j * G + gid) * D + kc * 16 + 4 * tig) * 2);
        qa[kc][0] = x.x;
        qa[kc][1] = x.y;
      }
      // order these reads before the next segment's bulk copy (async proxy) into the slot
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.q_empty[qs]);
      ++q_n;
      const float c_gid = (F16 ? 1.f : row_to_f16<KC>(qa)) * a.scale_log2;
      cq[0] = __shfl_sync(0xffffffffu, c_gid, 8 * tig);
      cq[1] = __shfl_sync(0xffffffffu, c_gid, 8 * tig + 4);
    }

    constexpr int TW = 32 * C::SUB;   // tokens of a warp
    constexpr int NI = TW / 8;        // of a lane
    const int tw0 = w * TW;           // the warp's first
    if (tw0 < count) {
      // e4m3 rows past the context may hold NaN codes, which a zero weight does not remove
      if (FMT == PA_Q8_E4M3 && tw0 + TW > count) {
        constexpr int CH = D / 16;
        for (int i = lane; i < TW * CH; i += 32) {
          const int t = tw0 + i / CH;
          if (t >= count)
            *reinterpret_cast<uint4*>(Vst + row_off(t) + (((ch0 + i % CH) ^ swizzle(t)) << 4)) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint32_t st_u = smem_base + (uint32_t)s * C::STAGE_BYTES;

      // scales of this lane's tokens tw0 + 8 i + gid, asked for before the product
      float kf[NI], vf[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int at = sc_off(tw0 + 8 * i + gid);
        kf[i] = *reinterpret_cast<const float*>(ksc + at);
        vf[i] = *reinterpret_cast<const float*>(vsc + at);
      }
      // ---- S^T = K Q^T: row tiles of 16 tokens; element 2 i + e: token 8 i + gid of the
      // tile, head 2 tig + e
      float sc[TW / 16][4];
#pragma unroll
      for (int h = 0; h < TW / 16; ++h) {
        sc[h][0] = sc[h][1] = sc[h][2] = sc[h][3] = 0.f;
        const int t = tw0 + 16 * h + (lane & 7) + (((lane >> 3) & 1) << 3);
        const uint32_t base = st_u + (uint32_t)row_off(t) + ((uint32_t)(hi ^ (sw & 1)) << 4);
#pragma unroll
        for (int p = 0; p < KC / 2; ++p) {
          uint32_t r[4];  // chunk 2p: tokens 0..7, 8..15; chunk 2p + 1
          ldsm_x4(r, base + (((uint32_t)p << 5) ^ sw_hi));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a0, a1, a2, a3;
            widen4<FMT, false>(r[2 * i], a0, a2);
            widen4<FMT, false>(r[2 * i + 1], a1, a3);
            mma_f16(sc[h], a0, a1, a2, a3, qa[2 * p + i][0], qa[2 * p + i][1]);
          }
        }
      }
      // ---- online softmax ---------------------------------------------------------------
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        // (__fmul_rn is not contracted: the maximum and the difference from it take the same
        // rounded score. Of an unrounded one the difference could be half a unit of the maximum's
        // last place above 0, which from 2^24 on is a weight that no fp16 number holds. The two
        // factors first: the product of codes and queries of 2^14 times a bf16 key's scale alone
        // could overflow)
        sc[i >> 1][2 * (i & 1)] = __fmul_rn(sc[i >> 1][2 * (i & 1)], kf[i] * cq[0]);
        sc[i >> 1][2 * (i & 1) + 1] = __fmul_rn(sc[i >> 1][2 * (i & 1) + 1], kf[i] * cq[1]);
      }
      if (tw0 + TW > count) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (tw0 + 8 * i + gid >= count) {
            sc[i >> 1][2 * (i & 1)] = sc[i >> 1][2 * (i & 1) + 1] = -INFINITY;
            vf[i] = 0.f;
          }
      }
      float top[2] = {-INFINITY, -INFINITY};
      uint32_t vtop = 0u;
#pragma unroll
      for (int h = 0; h < TW / 16; ++h) {
        top[0] = fmaxf(top[0], fmaxf(sc[h][0], sc[h][2]));
        top[1] = fmaxf(top[1], fmaxf(sc[h][1], sc[h][3]));
        vtop = max(vtop, max(__float_as_uint(vf[2 * h]) & 0x7fffffffu,
                             __float_as_uint(vf[2 * h + 1]) & 0x7fffffffu));
      }
      vtop = __reduce_max_sync(0xffffffffu, vtop);
      const int e_new = (int)(vtop >> 23) - 127;
      if (__any_sync(0xffffffffu, top[0] > m_run[0] || top[1] > m_run[1]) || e_new > e_run) {
        float grow = 1.f;
        if (e_new > e_run) {
          grow = e_run - e_new < -126 ? 0.f : pow2f(e_run - e_new);
          e_run = e_new;
        }
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int m = 4; m < 32; m <<= 1)
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], m));
          const float m_new = fmaxf(m_run[e], top[e]);
          // (-inf only where every score so far is NaN)
          alpha[e] = m_new == m_run[e] ? 1.f : fast_exp2(m_run[e] - m_new);
          m_run[e] = m_new;
          m_ref[e] = m_new == -INFINITY ? 0.f : m_new;
          l_part[e] *= alpha[e];
          alpha[e] *= grow;
        }
#pragma unroll
        for (int n = 0; n < KC; ++n) {
          o[n][0] *= alpha[0];
          o[n][1] *= alpha[1];
          o[n][2] *= alpha[0];
          o[n][3] *= alpha[1];
        }
      }
      const float nu = pow2f(14 - e_run);
      // the operand's words, and what they lose: head gid, tokens 8 i + 2 tig, + 1
      uint32_t wt[NI], wl[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float p0 = fast_exp2(sc[i >> 1][2 * (i & 1)] - m_ref[0]);
        const float p1 = fast_exp2(sc[i >> 1][2 * (i & 1) + 1] - m_ref[1]);
        l_part[0] += p0;
        l_part[1] += p1;
        vf[i] *= nu;
        const float w0 = p0 * vf[i], w1 = p1 * vf[i];
        const uint32_t hi = f2_elt2<true>(w0, w1);
        wt[i] = transpose8(hi);
        const float2 held = f16x2_f2(hi);
        wl[i] = transpose8(f2_elt2<true>(w0 - held.x, w1 - held.y));
      }
      // ---- O^T += V^T W^T: blocks of 16 tokens ----------------------------------------
#pragma unroll
      for (int h = 0; h < TW / 16; ++h) {
        const int t = tw0 + 16 * h + (lane & 7) + (((lane >> 3) & 1) << 3);
        const uint32_t base =
            st_u + C::KV_BYTES + (uint32_t)row_off(t) + ((uint32_t)(hi ^ (sw & 1)) << 4);
#pragma unroll
        for (int p = 0; p < KC / 2; ++p) {
          uint32_t r[4];  // chunk 2p: tokens 0..7, 8..15; chunk 2p + 1
          ldsm_x4_t(r, base + (((uint32_t)p << 5) ^ sw_hi));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a0, a1, a2, a3;
            widen4<FMT, true>(r[2 * i], a0, a1);
            widen4<FMT, true>(r[2 * i + 1], a2, a3);
            mma_f16(o[2 * p + i], a0, a1, a2, a3, wt[2 * h], wt[2 * h + 1]);
            mma_f16(o[2 * p + i], a0, a1, a2, a3, wl[2 * h], wl[2 * h + 1]);
          }
        }
      }
    }

    if (flags & kFlagLast) {
      // ---- finalize the segment: from the warp's reference scale back to the values' ------
      const float back = pow2f(e_run - 14);
#pragma unroll
      for (int n = 0; n < KC; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] *= back;
      float l_all[2] = {l_part[0], l_part[1]};
#pragma unroll
      for (int m = 4; m < 32; m <<= 1) {
        l_all[0] += __shfl_xor_sync(0xffffffffu, l_all[0], m);
        l_all[1] += __shfl_xor_sync(0xffffffffu, l_all[1], m);
      }
      // several warps per KV head: merge their softmax states through the stage's K/V
      // shared memory once every consumer warp is done with it
      if constexpr (C::WPH > 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.seg_bar);
        if (!mbar_wait(&ctl.seg_bar, (uint32_t)(seg_count & 1), abort_flag)) gave_up();
      }
      float* merge = reinterpret_cast<float*>(Kst) + (size_t)j * (C::WPH - 1) * C::MERGE_FLOATS;
      if (w != 0) {
        float* mine = merge + (size_t)(w - 1) * C::MERGE_FLOATS;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int head = 2 * tig + e;
          if (head < G) {
#pragma unroll
            for (int n = 0; n < KC; ++n)
              *reinterpret_cast<float2*>(mine + head * D + n * 16 + 2 * gid) =
                  make_float2(o[n][e], o[n][2 + e]);
            if (gid == 0) {
              mine[kTcGMax * D + head] = m_run[e];
              mine[kTcGMax * D + kTcGMax + head] = l_all[e];
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.merge_bar[j]);
      } else {
        if constexpr (C::WPH > 1) {
          if (!mbar_wait(&ctl.merge_bar[j], (uint32_t)(seg_count & 1), abort_flag)) gave_up();
        }
        for (int w2 = 1; w2 < C::WPH; ++w2) {
          const float* other = merge + (size_t)(w2 - 1) * C::MERGE_FLOATS;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int head = 2 * tig + e;
            if (head < G) {
              const float m2 = other[kTcGMax * D + head];
              const float l2 = other[kTcGMax * D + kTcGMax + head];
              const float mm = fmaxf(m_run[e], m2);
              // (a state without scores, or with NaN alone, keeps what it has: 0 or NaN)
              const float a1 = m_run[e] == mm ? 1.f : fast_exp2(m_run[e] - mm);
              const float a2 = m2 == mm ? 1.f : fast_exp2(m2 - mm);
#pragma unroll
              for (int n = 0; n < KC; ++n) {
                const float2 ov =
                    *reinterpret_cast<const float2*>(other + head * D + n * 16 + 2 * gid);
                o[n][e] = o[n][e] * a1 + ov.x * a2;
                o[n][2 + e] = o[n][2 + e] * a1 + ov.y * a2;
              }
              l_all[e] = l_all[e] * a1 + l2 * a2;
              m_run[e] = mm;
            }
          }
        }
        // normalise and write the rows, or the partials for the combine (a NaN sum stays NaN)
        const int b = meta.b;
        const bool whole = (flags & kFlagWhole) != 0;
        const int slot = (ctl.x0 < meta.pb) ? 1 : 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int head = 2 * tig + e;
          if (head >= G) continue;
          const int hg = kvh * G + head;
          const float inv = l_all[e] == 0.f ? 0.f : 1.f / l_all[e];
          if (whole) {
            uint16_t* dst = static_cast<uint16_t*>(a.out) + ((int64_t)b * H + hg) * D + 2 * gid;
#pragma unroll
            for (int n = 0; n < KC; ++n) {
              const float r0 = o[n][e] * inv, r1 = o[n][2 + e] * inv;
              *reinterpret_cast<uint32_t*>(dst + n * 16) = f2_elt2<F16>(r0, r1);
            }
          } else {
            float* dst = a.part_o + (((int64_t)c * 2 + slot) * H + hg) * D + 2 * gid;
#pragma unroll
            for (int n = 0; n < KC; ++n)
              *reinterpret_cast<float2*>(dst + n * 16) = make_float2(o[n][e] * inv, o[n][2 + e] * inv);
            if (gid == 0)
              a.part_lse[((int64_t)c * 2 + slot) * H + hg] =
                  l_all[e] == 0.f ? -INFINITY : m_run[e] + fast_log2(l_all[e]);
          }
        }
        if (!whole) {
          __threadfence();
          __syncwarp();
          int old = 0;
          int* counter = a.counters + (int64_t)b * Hk + kvh;
          if (lane == 0) old = atomicAdd(counter, 1);
          old = __shfl_sync(0xffffffffu, old, 0);
          const int64_t nt = ctl.nt, pb = meta.pb;
          const int g = ctl.g_eff;
          const int64_t c_lo = cta_of(pb, nt, g);
          const int64_t c_hi = cta_of(pb + meta.nb - 1, nt, g);
          const int nseg = (int)(c_hi - c_lo + 1);
          if (old == nseg - 1) {  // last arrival: combine the partials of sequence b in CTA order
            __threadfence();
            const bool first_slot = tile_begin(c_lo, nt, g) < pb;
            uint16_t* dst = static_cast<uint16_t*>(a.out) + ((int64_t)b * H + kvh * G) * D;
            combine_q8<D, F16>(a.part_o, a.part_lse, dst, H, kvh * G, G, (int)c_lo, nseg, first_slot,
                               lane);
            if (lane == 0) *counter = 0;  // leave the counter zero for the next call
          }
        }
      }
      ++seg_count;
      reset();  // here, so that none of it is kept across the combine
      fence_proxy_async_smem();
    }
    // order this tile's shared-memory reads before the producer's next copy into the stage
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.empty[s]);
  }
}

template <int HS, int D, int FMT, bool F16>
int launch_decode_q8_t(DecodeQ8Args a, const DeviceInfo& info, cudaStream_t stream) {
  using C = Q8Cfg<HS, D>;
  static std::atomic<bool> attr_done[64];  // zero-initialised: false
  const int dev = info.device;
  if (dev < 0 || dev >= 64) return PA_ERR_CUDA;
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(paged_decode_q8_kernel<HS, D, FMT, F16>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM) != cudaSuccess)
      return PA_ERR_CUDA;
    attr_done[dev].store(true, std::memory_order_release);
  }
  int tb = tc_box_tokens(a.block_size, C::T);
  if (tb > 256) tb = 256;  // a box's largest extent
  Q8Maps tm;
  memset(&tm, 0, sizeof(tm));
  if (tb > 0 &&
      (!make_codes_map(&tm.k, a.k_cache, a.num_kv_heads / C::HPR, C::ROW, a.block_size,
                       a.num_blocks, tb, HS / C::HPR) ||
       !make_codes_map(&tm.v, a.v_cache, a.num_kv_heads / C::HPR, C::ROW, a.block_size,
                       a.num_blocks, tb, HS / C::HPR) ||
       !make_scales_map(&tm.ks, a.k_scale, a.num_kv_heads, a.block_size, a.num_blocks, tb, HS) ||
       !make_scales_map(&tm.vs, a.v_scale, a.num_kv_heads, a.block_size, a.num_blocks, tb, HS)))
    return PA_ERR_CUDA;
  // the automatic grid: one resident wave over all slabs
  const int slabs = a.num_kv_heads / HS;
  if (a.auto_grid) a.grid_ctas = slabs < info.num_sms ? info.num_sms / slabs : 1;
  const dim3 grid((unsigned)a.grid_ctas, (unsigned)slabs);
  if (launch_dependent(paged_decode_q8_kernel<HS, D, FMT, F16>, grid, dim3(kThreads), C::SMEM, stream,
                       tm, a, tb) != cudaSuccess)
    return PA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D, int FMT, bool F16>
int dispatch_slab_q8(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream) {
  switch (decode_head_slab(a.num_kv_heads)) {
    case 8: return launch_decode_q8_t<8, D, FMT, F16>(a, info, stream);
    case 4: return launch_decode_q8_t<4, D, FMT, F16>(a, info, stream);
    case 2: return launch_decode_q8_t<2, D, FMT, F16>(a, info, stream);
    default: return launch_decode_q8_t<1, D, FMT, F16>(a, info, stream);
  }
}

}  // namespace
}  // namespace pa
