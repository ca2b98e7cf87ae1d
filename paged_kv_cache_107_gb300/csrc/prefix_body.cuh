// prefix_body.cuh — the shared part of pa_decode_shared on the tcgen05 tensor cores (the body of
// the CTAs that take it; shared_decode.cuh launches them beside those of the rests).
//
// What it computes: for every group g of sequences that hold the same first L keys, every
// query head h and sequence b of the group, over each of the key ranges S that the work is cut
// into, the normalised row and its log-sum-exp
//   o = sum_{t in S} 2^(x_t - lse) v_t,  lse = log2 sum_{t in S} 2^(x_t),  x_t = log2(e) scale q.k_t.
// shared_join.cu joins them with those of the sequence's own keys (decode_tc.cuh).
//
// Why it pays: a decode reads the shared keys once for each sequence. Here the rows of a
// group (n sequences x the G query heads of a KV head) are a dense matrix, so each shared
// key and value is read once for 128 or 256 of them: below about 256 rows the bytes of the
// prefix bound it, above the products do.
//
// Structure (that of prefill_kernel.cuh, whose constants and helpers it uses): TMA warps for
// K, V and Q, a warp that issues tcgen05.mma and two softmax warpgroups, one for each of two
// slots of accumulators in tensor memory.
//  * Work: the steps of all units (GroupWork) form one stream, cut into equal shares
//    whose bounds need not be those of units: a long prefix is spread over all of these CTAs
//    whatever the number of groups. A CTA's share is a list of segments, each a range of
//    steps of one unit.
//  * A unit with two row tiles takes each key tile for both slots (one load, two products). A
//    unit with one row tile would leave the second slot idle and its own chain of product,
//    softmax, product exposed; it gives the slots alternate key tiles instead, and the two
//    softmax states are joined when the segment ends, through tensor memory, each warpgroup
//    writing half of the dims.
//  * The softmax sums, the running maxima and O stay in fp32; P is rounded to the element type
//    for the second product, as in the prefill.
#pragma once

#include "prefill_kernel.cuh"
#include "shared_groups.cuh"

namespace pa {
namespace {

template <int D>
struct PrefixCfg {
  // ring depths: 160 KB of K and V tiles at both head dims
  static constexpr int KS = D == 64 ? 4 : 2;
  static constexpr int VS = D == 64 ? 6 : 3;
  static constexpr int kTile = (D / 64) * kHalf;
};

// A range of steps of one unit (n = 0: the end of the share).
struct PrefixSeg {
  int first, n;  // the group's sequences
  int len;       // shared keys
  int nt;        // key tiles
  int pair, j;   // row tiles 2*pair (and 2*pair + 1 when two), KV head
  int s0, s1;    // steps
  int two;       // both slots take the same key tile
  // key tiles of slot g: tile(g, it) for it < count(g)
  __device__ __forceinline__ int steps() const { return s1 - s0; }
  __device__ __forceinline__ int tile(int g, int it) const {
    return two ? s0 + it : 2 * (s0 + it) + g;
  }
  __device__ __forceinline__ int count(int g) const {
    return two || g == 0 ? s1 - s0 : min(s1, nt >> 1) - s0;
  }
  __device__ __forceinline__ int tiles() const {  // K (or V) tiles loaded
    return two ? s1 - s0 : count(0) + max(0, count(1));
  }
};

// Segments on their way from the warp that works them out to the other roles.
constexpr int kSegSlots = 4;
constexpr int kSegReaders = 3 + 8;  // warps: V, MMA, Q, the softmax's
constexpr int kVWarp = 11;          // beside kTmaWarp (here K's), kMmaWarp and kQWarp

template <int D>
struct PrefixCtl {
  using C = PrefixCfg<D>;
  uint64_t q_full[2], q_empty[2];  // [row tile]
  uint64_t k_full[C::KS], k_empty[C::KS];
  uint64_t v_full[C::VS], v_empty[C::VS];
  uint64_t s_full[2], p_full[2], o_done[2];  // [slot]
  uint64_t seg_full[kSegSlots], seg_empty[kSegSlots];
  uint64_t join_there, join_back, join_read;
  uint32_t tmem_base;
  int abort;
  PrefixSeg segs[kSegSlots];
  float2 join[kRows];  // [row] slot 1's softmax maximum and sum, then the factors of both O
};

template <int D>
struct PrefixTiles {
  using C = PrefixCfg<D>;
  unsigned char q[2][C::kTile];
  unsigned char k[C::KS][C::kTile];
  unsigned char v[C::VS][C::kTile];
};

constexpr int kPrefixCtlBytes = 1616;

template <int D>
constexpr size_t prefix_smem_bytes() {
  return 1023 + kPrefixCtlBytes + sizeof(PrefixTiles<D>);
}

// a / b, in 32 bits where both fit (a 64-bit division is a long subroutine).
__device__ __forceinline__ uint64_t quotient(uint64_t a, uint64_t b) {
  return ((a | b) >> 32) == 0 ? (uint64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Hands out a CTA's segments in order.
struct PrefixWalk {
  int64_t x, x1;  // next step, end of the share
  int64_t gx;     // first step of group g
  int g;
  int first, n, prefix;

  __device__ __forceinline__ void load_group(const SharedArgs& sh) {
    first = __ldg(sh.group_starts + g);
    n = __ldg(sh.group_starts + g + 1) - first;
    prefix = __ldg(sh.prefix_lens + g);
  }
  __device__ __forceinline__ bool next(PrefixSeg& s, const SharedArgs& sh, int Hk, int P) {
    while (x < x1) {
      GroupWork w(sh, n, prefix, P);
      while (x - gx >= w.steps(Hk) && g + 1 < sh.num_groups) {
        gx += w.steps(Hk);
        ++g;
        load_group(sh);
        w = GroupWork(sh, n, prefix, P);
      }
      const uint64_t rel = (uint64_t)(x - gx), per_pair = (uint64_t)Hk * (kUnitSteps + w.nt);
      const uint64_t pair = min(quotient(rel, per_pair), (uint64_t)w.full);
      const uint64_t in_pair = rel - pair * per_pair;
      const uint32_t us = (uint32_t)w.unit_steps((int)pair);
      const uint64_t unit = quotient(in_pair, us);
      const int v0 = (int)(in_pair - unit * us);
      const int v1 = (int)min((int64_t)us, (int64_t)v0 + (x1 - x));
      x += v1 - v0;
      if (v1 <= kUnitSteps) continue;  // nothing but the start's share
      s.first = first;
      s.n = n;
      s.len = prefix;
      s.nt = w.nt;
      s.pair = (int)pair;
      s.two = (int)pair < w.full;
      s.j = (int)unit;
      s.s0 = max(0, v0 - kUnitSteps);
      s.s1 = v1 - kUnitSteps;
      return true;
    }
    return false;
  }
};

template <int D>
__device__ __forceinline__ void note_timeout(PrefixCtl<D>& c, int* dev_err) {
  c.abort = 1;
  set_dev_err(dev_err, PA_DEV_ERR_TIMEOUT);
}

// 32 consecutive floats, one full 32-byte sector per store (p 32-byte aligned).
__device__ __forceinline__ void store32(float* p, const float* v) {
#pragma unroll
  for (int e = 0; e < 32; e += 8)
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + e), "f"(v[e]),
                 "f"(v[e + 1]), "f"(v[e + 2]), "f"(v[e + 3]), "f"(v[e + 4]), "f"(v[e + 5]),
                 "f"(v[e + 6]), "f"(v[e + 7])
                 : "memory");
}

template <int D, bool F16>
__device__ __forceinline__ void prefix_body(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                            const CUtensorMap& tm_q, const DecodeSharedArgs& a,
                                            const int box_rows, unsigned char* smem_raw,
                                            const SharedPlan& plan, int active_ctas) {
  using C = PrefixCfg<D>;
  using Ctl = PrefixCtl<D>;
  static_assert(sizeof(Ctl) <= kPrefixCtlBytes, "control block");
  constexpr int NH = D / 64;
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem_raw);
  PrefixTiles<D>& sm = *reinterpret_cast<PrefixTiles<D>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + kPrefixCtlBytes + 1023) & ~uintptr_t(1023));

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int H = a.num_heads, Hk = a.num_kv_heads, G = H / Hk;
  const int P = kRows / G;  // sequences per row tile (rows P*G..127 are padding)
  const SharedArgs& sh = a.sh;

  if (tid == 0) {
    for (int g = 0; g < 2; ++g) {
      mbar_init(&ctl.q_full[g], 1);
      mbar_init(&ctl.q_empty[g], 1);
      mbar_init(&ctl.s_full[g], 1);
      mbar_init(&ctl.p_full[g], kRows);
      mbar_init(&ctl.o_done[g], 1);
    }
    for (int s = 0; s < C::KS; ++s) {
      mbar_init(&ctl.k_full[s], 1);
      mbar_init(&ctl.k_empty[s], 1);
    }
    for (int s = 0; s < C::VS; ++s) {
      mbar_init(&ctl.v_full[s], 1);
      mbar_init(&ctl.v_empty[s], 1);
    }
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(&ctl.seg_full[i], 1);
      mbar_init(&ctl.seg_empty[i], kSegReaders);
      ctl.segs[i].n = 0;
    }
    mbar_init(&ctl.join_there, kRows);
    mbar_init(&ctl.join_back, kRows);
    mbar_init(&ctl.join_read, 2 * kRows);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    umma::tmem_alloc(&ctl.tmem_base, kTmemCols);
    umma::tmem_relinquish();
  }
  // this CTA's share of the steps, and the group of the first: the last one that starts at it
  // or before
  PrefixWalk walk{prefix_begin(blockIdx.x, plan.nx, plan.prefix_ctas),
                  prefix_begin(blockIdx.x + 1, plan.nx, plan.prefix_ctas), 0, 0, 0, 0, 0};
  {
    int lo = 0, hi = sh.num_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (plan.first_x[mid] <= walk.x) lo = mid;
      else hi = mid - 1;
    }
    walk.g = lo;
    walk.gx = plan.first_x[lo];
    walk.first = plan.starts[lo];
    walk.n = plan.starts[lo + 1] - walk.first;
    walk.prefix = plan.prefix[lo];
  }
  // every grid before this one is complete from here on: q and the caches may be read and the
  // workspace written
  pdl_wait();
  write_prefix_parts(a, plan, active_ctas, kPrefillThreads);
  // the plan's arrays lie where copies land next, written through the generic proxy
  fence_proxy_async_smem();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  volatile int* abort_flag = &ctl.abort;
  PrefixSeg seg;
  int seg_n = 0;  // segments read
  // The next segment into s (a whole warp calls it); false at the end, and after a wait that
  // ran out: a slot is read only when it is full and (below) written only when it is empty.
  auto next_seg = [&](PrefixSeg& s) {
    const int slot = seg_n % kSegSlots;
    const bool there = mbar_wait(&ctl.seg_full[slot], (uint32_t)((seg_n / kSegSlots) & 1), abort_flag);
    if (!__all_sync(0xffffffffu, there)) {
      note_timeout(ctl, a.dev_err);
      return false;
    }
    ++seg_n;
    s = ctl.segs[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.seg_empty[slot]);
    return s.n != 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == kTmaWarp || warp == kVWarp) {
      // ---------------------------------------------------------------- TMA producers
      // One warp for K, one for V: at small block sizes a tile takes many boxes, and the warp
      // that issues them is what a step waits for (16 steps of a lone row tile at block size
      // 16, head_dim 64: 44 us with one warp for both). Lane b owns box b of a tile (box_rows
      // keys of one block). The K warp also works out the segments and hands them on.
      const bool is_v = warp == kVWarp;
      const int bs = a.block_size;
      const int boxes = kKeys / box_rows;
      const int stages = is_v ? C::VS : C::KS;
      uint64_t* const empty = is_v ? ctl.v_empty : ctl.k_empty;
      uint64_t* const full = is_v ? ctl.v_full : ctl.k_full;
      unsigned char* const ring = is_v ? sm.v[0] : sm.k[0];
      const CUtensorMap* const map = is_v ? &tm_v : &tm_k;
      int cnt = 0;  // tiles loaded
      int pub = 0;  // segments handed on
      auto my_next_seg = [&](PrefixSeg& t) {
        if (is_v) return next_seg(t);
        const bool more = walk.next(t, sh, Hk, P);
        if (!more) t.n = 0;
        const int slot = pub % kSegSlots;
        bool free = true;
        if (lane == 0) {
          free = pub < kSegSlots || mbar_wait(&ctl.seg_empty[slot],
                                              (uint32_t)(((pub / kSegSlots) - 1) & 1), abort_flag);
          if (free) {
            ctl.segs[slot] = t;
            mbar_arrive(&ctl.seg_full[slot]);
          } else {
            note_timeout(ctl, a.dev_err);
          }
        }
        ++pub;
        return __all_sync(0xffffffffu, free) && more;
      };
      // this lane's block id of a key tile: -1 past the prefix, -2 out of the pool
      auto read_id = [&](const PrefixSeg& t, int tile) {
        const int key0 = tile * kKeys + lane * box_rows;
        if (lane >= boxes || key0 >= t.len) return -1;
        const int id = __ldg(a.block_tables + (int64_t)t.first * a.max_blocks + key0 / bs);
        return id >= 0 && (int64_t)id < a.num_blocks ? id : -2;
      };
      auto load = [&](int j, int tile, int id) {
        const int st = cnt % stages;
        if (lane == 0 && cnt >= stages &&
            !mbar_wait(&empty[st], (uint32_t)(((cnt / stages) - 1) & 1), abort_flag))
          note_timeout(ctl, a.dev_err);
        ++cnt;
        if (!is_v && __any_sync(0xffffffffu, id == -2) && lane == 0)
          set_dev_err(a.dev_err, PA_DEV_ERR_BLOCK_ID);
        const uint32_t valid = __ballot_sync(0xffffffffu, id >= 0);
        if (lane == 0)
          mbar_arrive_expect_tx(&full[st], (uint32_t)__popc(valid) * NH * box_rows * 128u);
        __syncwarp();
        if (id >= 0) {
          const int row0 = (tile * kKeys + lane * box_rows) % bs;
          unsigned char* dst = ring + st * C::kTile + lane * box_rows * 128;
#pragma unroll
          for (int h2 = 0; h2 < NH; ++h2)
            umma::tma_load_4d(dst + h2 * kHalf, map, h2 * 64, row0, j, id, &full[st]);
        }
        __syncwarp();
      };
      // a step of the stream: the key tiles of both slots (two: one for both) and this lane's
      // block ids of them (read while the ring has no free slot)
      struct Step {
        int n, j;
        int tile[2], id[2];
      };
      bool more = my_next_seg(seg);
      int it = 0;
      auto next_step = [&]() {
        Step t{0, 0, {0, 0}, {-1, -1}};
        if (!more) return t;
        t.n = !seg.two && it < seg.count(1) ? 2 : 1;
        t.j = seg.j;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          t.tile[g] = seg.tile(g, it);
          if (g < t.n) t.id[g] = read_id(seg, t.tile[g]);
        }
        if (++it == seg.steps()) {
          more = my_next_seg(seg);
          it = 0;
        }
        return t;
      };
      Step cur = next_step();
      while (cur.n) {
#ifdef PA_TEST_DELAY_LAST_TILE_CYCLES
        // test build only: the wait for the K tiles of the CTA's last step runs out (the copies
        // are still issued, late, and awaited below)
        if (!is_v && !more) {
          const long long t_hold = clock64();
          while (clock64() - t_hold < (long long)(PA_TEST_DELAY_LAST_TILE_CYCLES)) {
          }
        }
#endif
        load(cur.j, cur.tile[0], cur.id[0]);
        if (cur.n == 2) load(cur.j, cur.tile[1], cur.id[1]);
        cur = next_step();
      }
      if (lane == 0) {  // the last copies land before the CTA may exit
        for (int c = cnt > stages ? cnt - stages : 0; c < cnt; ++c)
          mbar_wait_copies(&full[c % stages], (uint32_t)((c / stages) & 1));
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_s = umma::idesc_f32acc(kRows, kKeys, false, F16);
      constexpr uint32_t idesc_o = umma::idesc_f32acc(kRows, D, true, F16);
      int kc = 0, vc = 0;     // K and V tiles consumed
      int qc[2] = {0, 0};     // Q tiles consumed
      int pc[2] = {0, 0};     // P tiles consumed
      auto wait = [&](uint64_t* bar, int phase) {
        if (!mbar_wait(bar, (uint32_t)(phase & 1), abort_flag)) note_timeout(ctl, a.dev_err);
        umma::fence_after_sync();
      };
      auto commit1 = [&](uint64_t* bar) {
        if (elect_one()) umma::commit(bar);
        __syncwarp();
      };
      auto wait_k = [&]() { wait(&ctl.k_full[kc % C::KS], kc / C::KS); };
      auto wait_v = [&]() { wait(&ctl.v_full[vc % C::VS], vc / C::VS); };
      auto free_k = [&]() { commit1(&ctl.k_empty[kc++ % C::KS]); };
      auto free_v = [&]() { commit1(&ctl.v_empty[vc++ % C::VS]); };
      auto issue_s = [&](int g, int qt) {  // S_g = Q_qt K^T
        const uint64_t qd = umma::smem_desc(smem_u32(sm.q[qt]), 16, 1024);
        const uint64_t kd = umma::smem_desc(smem_u32(sm.k[kc % C::KS]), 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off16 = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
            umma::mma_bf16(tmem + col_s(g), qd + off16, kd + off16, idesc_s, kk > 0);
          }
          umma::commit(&ctl.s_full[g]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int g, bool first) {  // O_g (+)= P_g V
        const uint64_t vd = umma::smem_desc(smem_u32(sm.v[vc % C::VS]), kHalf, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            umma::mma_bf16_ts(tmem + col_o(g), tmem + col_s(g) + kk * 8,
                              vd + ((kk * 16 * 128) >> 4), idesc_o, !first || (kk > 0));
        }
        __syncwarp();
      };
      // the S products of step `it` (both slots), then its K tiles are free
      auto first_s = [&](const PrefixSeg& s) {
        wait(&ctl.q_full[0], qc[0]++);
        if (s.two) wait(&ctl.q_full[1], qc[1]++);
        wait_k();
        issue_s(0, 0);
        if (s.two) {
          issue_s(1, 1);
          free_k();
        } else {
          free_k();
          if (s.count(1) > 0) {
            wait_k();
            issue_s(1, 0);
            free_k();
          }
        }
        if (s.steps() == 1) {
          commit1(&ctl.q_empty[0]);
          if (s.two) commit1(&ctl.q_empty[1]);
        }
      };
      bool more = next_seg(seg);
      if (more) first_s(seg);
      while (more) {
        const int n = seg.steps();
        for (int it = 0; it < n; ++it) {
          if (seg.two) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              wait(&ctl.p_full[g], pc[g]++);
              if (g == 0) wait_v();
              issue_pv(g, it == 0);
              if (it == n - 1) commit1(&ctl.o_done[g]);
              if (it + 1 < n) {
                if (g == 0) wait_k();
                issue_s(g, g);
              }
            }
            free_v();
            if (it + 1 < n) free_k();
          } else {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if (it >= seg.count(g)) continue;
              wait(&ctl.p_full[g], pc[g]++);
              wait_v();
              issue_pv(g, it == 0);
              free_v();
              if (it == seg.count(g) - 1) commit1(&ctl.o_done[g]);
              if (it + 1 < seg.count(g)) {
                wait_k();
                issue_s(g, 0);
                free_k();
              }
            }
          }
          if (it + 2 == n) {  // the segment's last S products are issued
            commit1(&ctl.q_empty[0]);
            if (seg.two) commit1(&ctl.q_empty[1]);
          }
        }
        more = next_seg(seg);
        if (more) first_s(seg);
      }
    } else if (warp == kQWarp) {
      // ---------------------------------------------------------------- Q loader
      // P sequences x G heads of a row tile, one box per 64 dims; rows of the next group or
      // past the batch (zeros) land too and are never stored.
      int qn[2] = {0, 0};
      while (next_seg(seg)) {
        for (int qt = 0; qt < (seg.two ? 2 : 1); ++qt) {
          if (lane == 0) {
            if (qn[qt] > 0 &&
                !mbar_wait(&ctl.q_empty[qt], (uint32_t)((qn[qt] - 1) & 1), abort_flag))
              note_timeout(ctl, a.dev_err);
            mbar_arrive_expect_tx(&ctl.q_full[qt], (uint32_t)(P * G * D * 2));
#pragma unroll
            for (int h2 = 0; h2 < NH; ++h2)
              umma::tma_load_3d(sm.q[qt] + h2 * kHalf, &tm_q, h2 * 64, seg.j * G,
                                seg.first + (2 * seg.pair + qt) * P, &ctl.q_full[qt]);
          }
          ++qn[qt];
        }
      }
      if (lane == 0) {
        for (int qt = 0; qt < 2; ++qt)
          if (qn[qt] > 0) mbar_wait_copies(&ctl.q_full[qt], (uint32_t)((qn[qt] - 1) & 1));
      }
    }
    __syncwarp();
    umma::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
      umma::fence_after_sync();
      umma::tmem_dealloc(tmem, kTmemCols);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------------ softmax warpgroups
    const int g = warp >> 2;  // slot
    const int r = tid & 127;  // row == TMEM lane
    const int pos = r / G, hh = r % G;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    int sc = 0;             // S tiles of this slot consumed
    int oc[2] = {0, 0};     // o_done phases consumed, per slot
    int vbase = 0;          // V tiles of the earlier segments

    int jc = 0;  // segments whose slots were joined
    while (next_seg(seg)) {
      const int cnt = seg.count(g);
      float m_run = -INFINITY, l_run = 0.f;
      for (int it = 0; it < cnt; ++it) {
        if (!mbar_wait(&ctl.s_full[g], (uint32_t)(sc & 1), abort_flag)) note_timeout(ctl, a.dev_err);
        ++sc;
        umma::fence_after_sync();
        const int left = seg.len - seg.tile(g, it) * kKeys;  // keys of the tile that count
        if (left < kKeys) {
          // A prefix's last tile is masked where it lies. A branch that masks the row in registers
          // lengthened every tile: 116 against 112 us for 128 sequences behind 32,768 keys.
#pragma unroll 1
          for (int k0 = 0; k0 < kKeys; k0 += 32) {
            float y[32];
            umma::tmem_ld32(lane_addr + col_s(g) + k0, y);
            umma::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (k0 + c >= left) y[c] = -INFINITY;
            umma::tmem_st32(lane_addr + col_s(g) + k0, y);
          }
          umma::tmem_st_wait();
        }
        float sv[kKeys];
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) umma::tmem_ld32(lane_addr + col_s(g) + 32 * c4, sv + 32 * c4);
        umma::tmem_ld_wait();
        float mx[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mx[c] = sv[c];
#pragma unroll
        for (int c = 8; c < kKeys; ++c) mx[c & 7] = fmaxf(mx[c & 7], sv[c]);
        const float mt = a.scale_log2 * fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                              fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        // the running maximum only moves when it grows by more than 2^8 (then O is rescaled)
        float alpha = 1.f;
        bool rescale = false;
        if (it == 0) {
          m_run = mt;
        } else if (mt > m_run + kRescaleThreshold) {
          alpha = fast_exp2(m_run - mt);
          m_run = mt;
          rescale = true;
        }
        const float m_safe = m_run == -INFINITY ? 0.f : m_run;
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
        const float2 nm2 = make_float2(-m_safe, -m_safe);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < kKeys / 2; ++c) {
          const float2 x = umma::ffma2(make_float2(sv[2 * c], sv[2 * c + 1]), sc2, nm2);
          const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          acc[c & 3] = umma::fadd2(acc[c & 3], p);
          sv[c] = __uint_as_float(pack_elt2<F16>(p.x, p.y));
        }
        const float2 tt = umma::fadd2(umma::fadd2(acc[0], acc[1]), umma::fadd2(acc[2], acc[3]));
        l_run = l_run * alpha + (tt.x + tt.y);
        umma::tmem_st32(lane_addr + col_s(g), sv);
        umma::tmem_st32(lane_addr + col_s(g) + 32, sv + 32);
        if (__any_sync(0xffffffffu, rescale)) {  // S_g(it) completed after PV_g(it-1)
          float ob[32];
#pragma unroll
          for (int c4 = 0; c4 < D / 32; ++c4) {
            umma::tmem_ld32(lane_addr + col_o(g) + 32 * c4, ob);
            umma::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) ob[e] *= alpha;
            umma::tmem_st32(lane_addr + col_o(g) + 32 * c4, ob);
          }
        }
        if (left < kKeys) {  // rows of V past the prefix must not meet a zero probability
          const int vi = vbase + (seg.two ? it : 2 * it + g);
          const int st = vi % C::VS;
          if (!mbar_wait(&ctl.v_full[st], (uint32_t)((vi / C::VS) & 1), abort_flag))
            note_timeout(ctl, a.dev_err);
          if (r >= left) {
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch)
              *reinterpret_cast<uint4*>(sm.v[st] + (ch >> 3) * kHalf + r * 128 + (ch & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        umma::tmem_st_wait();
        umma::fence_before_sync();
        mbar_arrive(&ctl.p_full[g]);
      }
      vbase += seg.tiles();

      // ---- the segment's rows: O / l and the log-sum-exp ------------------------------
      const int tile = seg.two ? 2 * seg.pair + g : 2 * seg.pair;
      const int b = seg.first + tile * P + pos;
      const bool row_ok = pos < P && b < seg.first + seg.n;
      const int hq = seg.j * G + hh;
      float* dst;
      float* dst_lse;
      if (seg.s0 == 0) {
        dst = sh.first_o + ((int64_t)b * H + hq) * D;
        dst_lse = sh.first_lse + (int64_t)b * H + hq;
      } else {
        const int64_t at = (int64_t)blockIdx.x * 256 + (seg.two ? g * kRows : 0) + r;
        dst = sh.more_o + at * D;
        dst_lse = sh.more_lse + at;
      }
      auto wait_o = [&](int s) {
        if (!mbar_wait(&ctl.o_done[s], (uint32_t)(oc[s] & 1), abort_flag)) note_timeout(ctl, a.dev_err);
        ++oc[s];
      };
      if (seg.two) {
        wait_o(g);
        umma::fence_after_sync();
        const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
        if (row_ok) *dst_lse = l_run > 0.f ? m_run + fast_log2(l_run) : -INFINITY;
#pragma unroll
        for (int c4 = 0; c4 < D / 32; ++c4) {
          float ob[32];
          umma::tmem_ld32(lane_addr + col_o(g) + 32 * c4, ob);
          umma::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) ob[e] *= inv;
          if (row_ok) store32(dst + 32 * c4, ob);
        }
        // The other slot's phase is counted without a wait: where the next segment has one step,
        // its o_done can complete before a slower warpgroup here has looked, and the parity would
        // have come round. (A join, below, comes after the other warpgroup's own wait for it.)
        ++oc[1 - g];
      } else {
        // join the slots: warpgroup 1 hands over its maximum and sum, warpgroup 0 returns the
        // factors of both accumulators, and each takes half of the dims of both
        const bool has_b = seg.count(1) > 0;
        float fa, fb;
        if (g == 1) {
          ctl.join[r] = make_float2(m_run, l_run);
          mbar_arrive(&ctl.join_there);
          if (!mbar_wait(&ctl.join_back, (uint32_t)(jc & 1), abort_flag))
            note_timeout(ctl, a.dev_err);
          fa = ctl.join[r].x;
          fb = ctl.join[r].y;
        } else {
          if (!mbar_wait(&ctl.join_there, (uint32_t)(jc & 1), abort_flag))
            note_timeout(ctl, a.dev_err);
          const float2 ml = ctl.join[r];  // (-inf, 0) without a tile
          const float m = fmaxf(m_run, ml.x);
          fa = m == -INFINITY ? 0.f : fast_exp2(m_run - m);
          fb = m == -INFINITY ? 0.f : fast_exp2(ml.x - m);
          const float l = l_run * fa + ml.y * fb;
          const float inv = l > 0.f ? 1.f / l : 0.f;
          if (row_ok) *dst_lse = l > 0.f ? m + fast_log2(l) : -INFINITY;
          fa *= inv;
          fb *= inv;
          ctl.join[r] = make_float2(fa, fb);
          mbar_arrive(&ctl.join_back);
        }
        wait_o(0);
        if (has_b) wait_o(1);
        umma::fence_after_sync();
#pragma unroll
        for (int c4 = 0; c4 < D / 64; ++c4) {
          const int col = g * (D / 2) + 32 * c4;
          float oa[32], ob[32];
          umma::tmem_ld32(lane_addr + col_o(0) + col, oa);
          if (has_b) umma::tmem_ld32(lane_addr + col_o(1) + col, ob);
          umma::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) oa[e] = oa[e] * fa + (has_b ? ob[e] * fb : 0.f);
          if (row_ok) store32(dst + col, oa);
        }
        // neither slot's O (nor join) is written again before both warpgroups have read them
        umma::fence_before_sync();
        mbar_arrive(&ctl.join_read);
        if (!mbar_wait(&ctl.join_read, (uint32_t)(jc & 1), abort_flag))
          note_timeout(ctl, a.dev_err);
        umma::fence_after_sync();
        ++jc;
      }
    }
    umma::fence_before_sync();
    __syncthreads();
  }
}

}  // namespace
}  // namespace pa
