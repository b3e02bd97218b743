// Attention of a ragged batch of new tokens over their pages (qsa_paged_prefill)
// on the 5th-generation tensor cores.
//
//   out[t][h] = sum_j softmax_j(q[t][h] . k[j] scale) v[j]
//
// over the keys j up to the token's own that window and sinks leave; one pass
// with a running maximum and sum.
//
// Item = (128 query rows of one sequence, KV head); the rows are
// the sequence's (token, query head of the KV head) pairs laid out flat, so any
// head count fills the tiles and the heads of a KV head share its loads.  The
// keys that any row sees are numbered without the gap between sinks and window
// and taken in tiles of 128.  Persistent CTAs (one per SM) walk the items, those
// of the last tokens (the most keys) first.
//   * warps 0-7 (softmax): two warpgroups that take the tiles in turn, a thread a
//     query row (TMEM lane): mask, tile maximum, the running maximum from the
//     other group (raised only when a tile exceeds it by more than 8, so the
//     rescale of O is rare), handed back before the exponentials (base 2), then P
//     packed to 16 bits, for head dims 64 and 128 into TMEM columns of its own,
//     for 256 in place of the scores.  So one group's exponentials run beside the
//     other's loads and maxima.  At the end O / l and the log-sum-exp.
//   * warp 13 (K): slots of 128 keys x 64 dims by TMA, a box of 16 to 64 rows of
//     a page at a time (the numbering of the keys is rounded so that no box
//     crosses a page).  K rows that nobody sees need no care: their scores are
//     replaced.
//   * warps 8-11 (V): the Q tile, then slots of 128 * 64 / D keys x D dims by
//     cp.async, 16 bytes a thread; rows that no query sees, whose memory may hold
//     anything, are zero.  Page sizes that are no multiple of 16 have K this way
//     too.  K by one engine and V by the other because neither feeds the tensor
//     cores alone: a TMA box takes 52 + 3.2 cycles a row of 128 bytes (at most 40
//     bytes a cycle), four warps of cp.async bring 32.
//   * warp 12: S(i) = Q K^T (M = 128, N = 128); warp 14: O += P V (N = D).  Two
//     issuers, so a ready P V never waits behind the next S.
// Registers: 184 a softmax thread, 72 the others (setmaxnreg; 168 and 88: 4 % slower).
// Every mbarrier wait is bounded (timeout -> error word, clean exit): on an abort
// every role leaves its loop, the loaders wait for their own copies and the MMA
// thread for its last commit before TMEM is released.
//
// Balance: with few items their tiles, laid end to end, are cut evenly over the
// CTAs, so a short chunk over a long prefix and batches of any mix of lengths keep
// every SM busy.  A CTA's piece of an item that it shares goes to the scratch as
// normalised fp32 rows with their log-sum-exp; the join kernel adds the pieces in
// the order of the keys.  More items than MAX_EVEN, and pages that TMA cannot
// fetch, are dealt out whole: there one long sequence among short ones sets the
// time (may_cut below has the figures).
//
// Measured: 16384 tokens of 32 + 8 heads of 128 1.96 to 2.2 ms, 1000 to 1120 TFLOP/s;
// of 16 heads of 64 0.83 to 0.98 ms, 560 to 660 TFLOP/s (by GPU and clock).  Bound
// there by the exponentials: 128 x 128 of a tile take the special-function units 1024
// cycles, both products of 128 dims 1030, of 64 dims 515.  5 tokens of 64 sequences
// over 2000 to 30000 keys (24 + 2 heads of 256): 243 to 246 us, 5.6 TB/s of keys and
// values, 86 % of a copy's rate.
#include "paged_prefill.cuh"

namespace qsa {
namespace {

constexpr int M = 128;                              // query rows of an item
// Query rows of a sequence, on average, from which pairs are used: more than one
// tile of 128 (24 + 2 heads of 256, single against pairs: 11 tokens, 132 rows, over
// 80K keys 75 and 64 us; 21 tokens 78 and 71; 37 tokens 110 and 95; 8 x 37 over 20K
// 215 and 173; 16 x 30 over 1000 37 and 35; but 10 tokens, 120 rows, over 20K 32.5
// and 34.8).
constexpr int64_t PAIR_ROWS = 129;
constexpr int JOIN_CTAS = 592;                      // of the join: four to an SM
constexpr uint32_t SLOT = 16384;
constexpr int NS = 5;                               // slots of the K ring and of the V ring
constexpr uint32_t OFF_K = 65536;                   // Q: up to 128 rows x 512 B
constexpr uint32_t OFF_V = OFF_K + NS * SLOT;
constexpr uint32_t OFF_XCH = OFF_V + NS * SLOT;     // running maxima [2][128], row sums [2][128]
constexpr uint32_t OFF_OK = OFF_XCH + 2048;         // rows that are there, of NOK tiles, 32 bytes each
constexpr uint32_t OFF_BAR = OFF_OK + 32 * NOK;
constexpr uint32_t SMEM = OFF_BAR + 448;
static_assert(SMEM <= 232448, "prefill smem");

template <class E, int D, bool TMA, bool EVEN>
__global__ void __launch_bounds__(THREADS, 1) paged_prefill_kernel(const __grid_constant__ Args x) {
  constexpr int NCH = D / 64;                       // 64-dim chunks: K (and V) slots of a tile
  constexpr int KV = KT / NCH;                      // keys of a V slot
  constexpr int GR = NCH < 2 ? 1 : 2;               // slots to a "full" barrier
  constexpr uint32_t IDESC = umma_idesc_bf16_f32(M, KT) &
                             (std::is_same<E, __half>::value ? ~((1u << 7) | (1u << 10)) : ~0u);   // f16: 0
  constexpr uint32_t IDESC_PV = ((IDESC & ~(63u << 17)) | ((uint32_t)(D >> 3) << 17)) | (1u << 16);   // V MN-major
  using X = Elem<E>;
  using TM = Tmem<D, false>;
  const PagedAttnArgs& a = x.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* k_full = bars;                          // [NS]
  uint64_t* k_empty = k_full + NS;                  // [NS]
  uint64_t* v_full = k_empty + NS;                  // [NS]
  uint64_t* v_empty = v_full + NS;                  // [NS]
  uint64_t* q_full = v_empty + NS;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;                   // [2]
  uint64_t* s_empty = s_full + 2;                   // [2] (P apart from S)
  uint64_t* p_full = s_empty + 2;                   // [2]
  uint64_t* pv_done = p_full + 2;                   // [2]
  uint64_t* o_empty = pv_done + 2;
  uint64_t* hand = o_empty + 1;                     // [2][4]: the maximum after a tile, 32 rows each
  uint64_t* turn = hand + 8;                        // [2][4]: the exponentials of a tile
  uint64_t* xbar = turn + 8;                        // [4]: row sums, 32 rows each
  uint64_t* mma_done = xbar + 4;                    // [2]: the S and the P V issuer
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // the shuffle tells the compiler that a warp has one role
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (tid == 0) report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&k_full[s], TMA ? GR : LWARPS);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], LWARPS);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(q_full, LWARPS);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 4); mbar_init(&p_full[i], 4); mbar_init(&pv_done[i], 1); }
    for (int i = 0; i < 8; ++i) { mbar_init(&hand[i], 1); mbar_init(&turn[i], 1); }
    mbar_init(o_empty, 8);
    for (int i = 0; i < 4; ++i) mbar_init(&xbar[i], 2);
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) { tmem_alloc(tmem_slot, TMEM_COLS); tmem_relinquish(); }
  if (EVEN) pdl_launch();                           // the join follows
  tc_fence_before();
  // (without EVEN the walk is of launch constants, not through a structure that
  // the roles' loops would have to read)
  Walk walk{};
  if constexpr (EVEN) walk = uniform(make_walk<M>(x, blockIdx.x, gridDim.x, smem));   // in Q's place
  const ItemNo<EVEN> w_first = EVEN ? walk.w : blockIdx.x, w_step = EVEN ? walk.step : gridDim.x;
  const ItemNo<EVEN> w_last = EVEN ? walk.last : x.n_slots * x.a.hk - 1;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t per = (uint32_t)a.hq / (uint32_t)a.hk;

  if (warp >= W_LOAD) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
  if (warp >= W_LOAD && warp < W_MMA) {
    // ------------------------------------------- Q and V (and K without TMA)
    const int lt = tid - 32 * W_LOAD, c = lt & 7, rt = lt >> 3;   // 16-byte chunk, row of a pass
    const int lw = warp - W_LOAD;
    int kslot = 0, vslot = 0, kgrp = 0, vgrp = 0;                 // slot, and barrier of its group
    uint32_t keph = 1, veph = 1, items_done = 0, count = 0;       // count: K tiles so far
    bool ok = true;
    // after the copies of this thread: full once every warp's have landed
    auto done = [&](uint64_t* bar) {
      cp_async_hold(bar);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    for (ItemNo<EVEN> w = w_first; ok && w <= w_last; w += w_step) {
      const Item<M> it = item_of<M, EVEN>(x, walk, w);
      if (it.n_tiles <= 0) continue;
      const int32_t* table = a.kv.table + (int64_t)it.b * a.kv.table_ld;
      const int64_t head = (int64_t)it.g * a.kv.head_stride + 8 * c;
      auto key_of = [&](int v) { return v < it.ns ? v : it.lo + (v - it.ns); };
      // A tile's rows: offset of this thread's chunk, and whether the row is there
      // (some query sees it and its page is one).
      struct Rows { int64_t off[RJ]; uint32_t ok; };
      // Page ids are loaded a tile ahead, all at once.  With TMA the 16 rows of a
      // pass lie in one page (page size and numbering are multiples of 16): lane j
      // finds pass j, the others take its place by a shuffle.  Else each thread
      // finds its rows rt + RT j.
      constexpr int NI = TMA ? 1 : RJ;
      int ids[NI];
      const int pass = lane % RJ;
      auto load_ids = [&](int tile) {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int v = tile * KT + (TMA ? RT * pass : RT * j + rt);
          const int key = key_of(max(min(v, it.n_vis - 1), 0));
          ids[j] = __ldg(table + page_of(a.kv, (uint32_t)min(key, a.kv.capacity - 1)));
        }
      };
      auto in_page = [&](int key) -> int64_t {
        return (int64_t)(key - (int)(page_of(a.kv, (uint32_t)key) * (uint32_t)a.kv.page_size)) * a.kv.token_stride;
      };
      auto needed = [&](int v, int key) { return v < it.n_vis && (key >= it.first || key < a.sinks); };
      const int64_t mine = head + (int64_t)rt * a.kv.token_stride;
      auto find_rows = [&](int tile, Rows& d) {
        d.ok = 0;
        if constexpr (TMA) {
          const int v = tile * KT + RT * pass, key = key_of(v);
          const bool any = v < it.n_vis && (key + RT > it.first || key < a.sinks);
          const bool good = any && (uint32_t)ids[0] < (uint32_t)a.kv.n_pages;
          if (any && !good) report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
          const bool clean = good && v + RT <= it.n_vis && (key >= it.first || key + RT <= a.sinks);
          const int64_t off = good ? (int64_t)ids[0] * a.kv.page_stride + in_page(key) : 0;
#pragma unroll
          for (int j = 0; j < RJ; ++j) d.off[j] = __shfl_sync(0xffffffffu, off, j) + mine;
          if (__all_sync(0xffffffffu, clean)) {
            d.ok = (1u << RJ) - 1;
          } else {
            const uint32_t there = __ballot_sync(0xffffffffu, good);
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
              const int r = tile * KT + RT * j + rt;
              const bool ok = (there >> j & 1) && needed(r, key_of(r));
              d.ok |= (uint32_t)ok << j;
            }
          }
        } else {
          bool bad = false;
#pragma unroll
          for (int j = 0; j < RJ; ++j) {
            const int v = tile * KT + RT * j + rt, key = key_of(v);
            const bool want = needed(v, key), good = want && (uint32_t)ids[j] < (uint32_t)a.kv.n_pages;
            d.off[j] = good ? (int64_t)ids[j] * a.kv.page_stride + in_page(key) + head : 0;
            d.ok |= (uint32_t)good << j;
            bad |= want && !good;
          }
          if (bad) report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
        }
      };
      const uint32_t lane_dst = swz128(rt, c);         // rows of a pass are 16 apart: the same swizzle in each
      auto load_k = [&](const Rows& d) -> bool {
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          // the warp's four rows of the pass: one byte of their bits
          const uint32_t bits = __ballot_sync(0xffffffffu, (d.ok >> j & 1) && c == 0);
          if (lane == 0) {
            const uint32_t four = (bits & 1) | (bits >> 7 & 2) | (bits >> 14 & 4) | (bits >> 21 & 8);
            reinterpret_cast<volatile uint8_t*>(smem + OFF_OK)[(count % NOK) * 32 + j * LWARPS + lw] = (uint8_t)four;
          }
        }
        ++count;
        for (int ch = 0; ch < NCH; ++ch) {
          if (!bar_wait(&k_empty[kslot], keph, abort_flag, a.err)) return false;
          const uint32_t dst = smem_u32(smem + OFF_K + kslot * SLOT) + lane_dst;
#pragma unroll
          for (int j = 0; j < RJ; ++j)
            cp_async16_zfill(dst + RT * j * 128, a.kv.k + d.off[j] + 64 * ch, d.ok >> j & 1);
          if (ch % GR == GR - 1) {
            done(&k_full[kgrp]);
            if (++kgrp == NS) kgrp = 0;
          }
          if (++kslot == NS) { kslot = 0; keph ^= 1; }
        }
        return true;
      };
      auto load_v = [&](const Rows& d) -> bool {
#pragma unroll
        for (int s = 0; s < NCH; ++s) {
          if (!bar_wait(&v_empty[vslot], veph, abort_flag, a.err)) return false;
          const uint32_t dst = smem_u32(smem + OFF_V + vslot * SLOT) + lane_dst;
#pragma unroll
          for (int j = 0; j < KV / RT; ++j) {
            const uint16_t* src = a.kv.v + d.off[s * (KV / RT) + j];
            const bool there = d.ok >> (s * (KV / RT) + j) & 1;
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch) cp_async16_zfill(dst + ch * (KV * 128) + RT * j * 128, src + 64 * ch, there);
          }
          if (s % GR == GR - 1) {
            done(&v_full[vgrp]);
            if (++vgrp == NS) vgrp = 0;
          }
          if (++vslot == NS) { vslot = 0; veph ^= 1; }
        }
        return true;
      };
      auto load_q = [&]() -> bool {
        // once the previous item's last S has read its own
        if (items_done > 0 && !bar_wait(q_empty, (items_done - 1) & 1, abort_flag, a.err)) return false;
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          const int r = RT * j + rt;
          const bool valid = r < it.rows;
          const uint32_t f = it.row0 + (valid ? r : 0);
          const uint16_t* src = a.q + it.q_row(a, per, f) * D + 8 * c;
#pragma unroll
          for (int ch = 0; ch < NCH; ++ch)
            cp_async16_zfill(smem_u32(smem + ch * SLOT) + swz128(r, c), valid ? src + 64 * ch : a.q, valid);
        }
        done(q_full);
        return true;
      };
      load_ids(it.tile0);
      if constexpr (TMA) {
        ok = load_q();
        for (int i = 0; ok && i < it.n_tiles; ++i) {
          Rows d;
          find_rows(it.tile0 + i, d);
          load_ids(it.tile0 + i + 1);
          ok = load_v(d);
        }
      } else {
        Rows d{};
        for (int i = 0; ok && i <= it.n_tiles; ++i) {
          const Rows before = d;
          if (i < it.n_tiles) {
            find_rows(it.tile0 + i, d);
            load_ids(it.tile0 + i + 1);
            ok = load_k(d);
          }
          if (ok) ok = i == 0 ? load_q() : load_v(before);
        }
      }
      ++items_done;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (TMA && warp == W_TMA) {
    // ---------------------------------------------------------------------- K
    int slot = 0, grp = 0;
    uint32_t eph = 1, gph = 0, count = 0;          // gph: parity of a group's barrier
    uint32_t landing = 0, open = 0;                // groups that copies went to; arrivals of an unfinished one
    bool ok = true;
    const int box = x.box, nb = KT / box;
    for (ItemNo<EVEN> w = w_first; ok && w <= w_last; w += w_step) {
      const Item<M> it = item_of<M, EVEN>(x, walk, w);
      if (it.n_tiles <= 0) continue;
      const int32_t* table = a.kv.table + (int64_t)it.b * a.kv.table_ld;
      // lane i has box i of a tile (lanes past the last repeat): its page, or -1
      // where no row of it is needed or the page is none, and its first row there
      auto find = [&](int tile, int& id, int& row) {
        const int v = tile * KT + (lane & (nb - 1)) * box, key = v < it.ns ? v : it.lo + (v - it.ns);
        const uint32_t pg = page_of(a.kv, (uint32_t)key);
        const bool any = v < it.n_vis && (key + box > it.first || key < a.sinks);
        id = any ? __ldg(table + pg) : -1;
        if (any && (uint32_t)id >= (uint32_t)a.kv.n_pages) {
          report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
          id = -1;
        }
        row = key - (int)(pg * (uint32_t)a.kv.page_size);
      };
      int id, row, id_n, row_n;
      find(it.tile0, id_n, row_n);
      for (int i = 0; ok && i < it.n_tiles; ++i) {
        id = id_n;
        row = row_n;
        const uint32_t good = __ballot_sync(0xffffffffu, id >= 0);
        reinterpret_cast<volatile uint8_t*>(smem + OFF_OK)[(count % NOK) * 32 + lane] = good >> (4 * lane / box) & 1 ? 15 : 0;
        __syncwarp();                              // every lane's bits before the arrival that lane 0 makes
        ++count;
        if (i + 1 < it.n_tiles) find(it.tile0 + i + 1, id_n, row_n);
        const bool mine = lane < nb && id >= 0;
        const uint32_t bytes = (uint32_t)__popc(good & ((1u << nb) - 1)) * box * 128;
        for (int ch = 0; ch < NCH; ++ch) {
          if (!__all_sync(0xffffffffu, bar_wait(&k_empty[slot], eph, abort_flag, a.err))) { ok = false; break; }
          if (lane == 0) {
            if (bytes) mbar_arrive_expect_tx(&k_full[grp], bytes);
            else mbar_arrive(&k_full[grp]);
          }
          __syncwarp();
          if (bytes) landing |= 1u << grp;
          open = (ch + 1) % GR;
          if (mine)
            tma_load_box(smem_u32(smem + OFF_K + slot * SLOT) + lane * box * 128, &x.tk, 64 * ch, row, it.g, id, &k_full[grp]);
          if (++slot == NS) { slot = 0; eph ^= 1; }
          if (ch % GR == GR - 1) {
            if (++grp == NS) { grp = 0; gph ^= 1; }
          }
        }
      }
    }
    // After an abort no TMA copy may still be writing when the CTA exits: wait
    // for the last phase of every group that copies went to (without an abort the
    // MMA waits for all of them).
    if (lane == 0) {
      if (open) mbar_arrive(&k_full[grp]);         // the group that an abort left half issued (GR = 2)
      for (int g = 0; g < NS; ++g)
        if (landing >> g & 1) mbar_wait_drain(&k_full[g], g < grp || (open && g == grp) ? gph : gph ^ 1, a.err);
    }
  } else if (warp == W_MMA) {
    // ---------------------------------------------------------------------- S
    int kslot = 0, kgrp = 0;
    uint32_t kph = 0, items_done = 0, count = 0;
    bool ok = true;
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, bar_wait(bar, parity, abort_flag, a.err));
    };
    for (ItemNo<EVEN> w = w_first; ok && w <= w_last; w += w_step) {
      const Item<M> it = item_of<M, EVEN>(x, walk, w);
      const int n_tiles = __shfl_sync(0xffffffffu, it.n_tiles, 0);
      if (n_tiles <= 0) continue;
      if (!wait(q_full, items_done & 1)) { ok = false; break; }
      fence_async_proxy();                          // Q: written by cp.async, read by the MMA
      for (int i = 0; i < n_tiles; ++i, ++count) {
        // S overwrites what the buffer had two tiles before: the scores, which are
        // in registers by now, or P in their place, whose P V is done.  (Either
        // barrier's next phase needs this S, so the parity is exact.)
        if (count >= 2 && !wait(TM::APART ? &s_empty[count & 1] : &pv_done[count & 1], ((count >> 1) - 1) & 1)) {
          ok = false;
          break;
        }
        const uint32_t d = tm + TM::s(count & 1);
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          if (ch % GR == 0) {
            if (!wait(&k_full[kgrp], kph)) { ok = false; break; }
            if (++kgrp == NS) { kgrp = 0; kph ^= 1; }
            if (!TMA) fence_async_proxy();
            tc_fence_after();
          }
          const uint32_t kb = base + OFF_K + kslot * SLOT;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_ss(d, desc_at(DESC_K, base + ch * SLOT + 32 * ks), desc_at(DESC_K, kb + 32 * ks), IDESC,
                    ch > 0 || ks > 0 ? 1u : 0u);
          umma_commit(&k_empty[kslot]);
          if (++kslot == NS) kslot = 0;
        }
        if (!ok) break;
#ifdef QSA_DEBUG_HOOKS
        // test hook: no CTA signals its first S, so the softmax times out
        if (!(a.inject == QSA_INJECT_PAGED_STALL && count == 0))
#endif
        umma_commit(&s_full[count & 1]);
        if (i == n_tiles - 1) umma_commit(q_empty);
      }
      ++items_done;
    }
    // every MMA of this warp has retired before TMEM is released (also after an
    // abort: a wait that ignores the flag)
    umma_commit(&mma_done[0]);
    mbar_wait_drain(&mma_done[0], 0, a.err);
  } else if (warp == W_PV) {
    // --------------------------------------------------------------------- PV
    int vslot = 0, vgrp = 0;
    uint32_t vph = 0, items_done = 0, count = 0;
    bool ok = true;
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, bar_wait(bar, parity, abort_flag, a.err));
    };
    for (ItemNo<EVEN> w = w_first; ok && w <= w_last; w += w_step) {
      const Item<M> it = item_of<M, EVEN>(x, walk, w);
      const int n_tiles = __shfl_sync(0xffffffffu, it.n_tiles, 0);
      if (n_tiles <= 0) continue;
      if (items_done > 0 && !wait(o_empty, (items_done - 1) & 1)) { ok = false; break; }
      for (int i = 0; i < n_tiles; ++i, ++count) {
        const uint32_t p = tm + TM::p(count & 1);
        if (!wait(&p_full[count & 1], (count >> 1) & 1)) { ok = false; break; }
#pragma unroll
        for (int s = 0; s < NCH; ++s) {
          if (s % GR == 0) {
            if (!wait(&v_full[vgrp], vph)) { ok = false; break; }
            if (++vgrp == NS) { vgrp = 0; vph ^= 1; }
            fence_async_proxy();                    // written by cp.async, read by the MMA
            tc_fence_after();
          }
          const uint32_t vb = base + OFF_V + vslot * SLOT;
#pragma unroll
          for (int ks = 0; ks < KV / 16; ++ks)
            umma_ts(tm + TM::O, p + 8 * (s * (KV / 16) + ks), desc_at(desc_mn(KV * 128), vb + 2048 * ks), IDESC_PV,
                    i > 0 || s > 0 || ks > 0 ? 1u : 0u);
          umma_commit(&v_empty[vslot]);
          if (++vslot == NS) vslot = 0;
        }
        if (!ok) break;
        umma_commit(&pv_done[count & 1]);
      }
      ++items_done;
    }
    umma_commit(&mma_done[1]);
    mbar_wait_drain(&mma_done[1], 0, a.err);
  } else if (warp < W_LOAD) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFT));
    softmax_role<E, D, M, false, EVEN>(x, smem, OFF_OK, OFF_XCH, {s_full, s_empty, p_full, pv_done, hand, turn, xbar, o_empty}, tmem, warp,
                                 lane, 0, walk, w_first, w_last, w_step, blockIdx.x, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the pieces of the items that are cut: S warps a query row (8 where the grid
// is large enough for all, down to one), each with every S-th piece, then the warps
// in order.  The grid fits the GPU at once, so a call without a cut item costs little
// beyond the launch.
template <class E, int D, int M>
__global__ void __launch_bounds__(256) paged_prefill_join_kernel(const __grid_constant__ Args x) {
  constexpr int W = D / 32;                         // dims of a lane: 2, 4 or 8
  constexpr int PER = MAX_EVEN / 8;                 // items that a warp looks at
  using X = Elem<E>;
  __shared__ float2 part[8][W / 2][32];
  __shared__ float2 ml[8];
  __shared__ int cut[MAX_EVEN], n_cut[8];
  const PagedAttnArgs& a = x.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_items = (int)(x.n_slots * a.hk);
  pdl_wait();
  const Scratch sc = scratch_of(a.scratch);
  // the cut items, in order
  uint32_t bits[PER / 32];
#pragma unroll
  for (int i = 0; i < PER / 32; ++i) {
    const int w = PER * warp + 32 * i + lane;
    bits[i] = __ballot_sync(0xffffffffu, w < n_items && sc.rec[min(w, MAX_EVEN - 1)].last >= 0);
  }
  int mine = 0;
#pragma unroll
  for (int i = 0; i < PER / 32; ++i) mine += __popc(bits[i]);
  if (lane == 0) n_cut[warp] = mine;
  __syncthreads();
  int at = 0, all = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < warp) at += n_cut[i];
    all += n_cut[i];
  }
#pragma unroll
  for (int i = 0; i < PER / 32; ++i) {
    if (bits[i] >> lane & 1) cut[at + __popc(bits[i] & ((1u << lane) - 1u))] = PER * warp + 32 * i + lane;
    at += __popc(bits[i]);
  }
  __syncthreads();
  int S = 8;
  while (S > 1 && all * (M / 8) * S > (int)gridDim.x) S >>= 1;
  const int blocks = M / 8 * S;                     // of an item
  for (int u = blockIdx.x; u < all * blocks; u += gridDim.x) {
    const int w = cut[u / blocks], sub = warp % S;
    const JoinRec rec = sc.rec[w];
    const Item<M> it(x, w);
    const int r = u % blocks * (8 / S) + warp / S;
    // pieces of this warp: sub, sub + S, ..
    const int n = r < it.rows ? (rec.last - rec.first + S - sub) / S : 0;
    auto row_of = [&](int i) {
      const int p = i * S + sub;
      return (int64_t)(2 * (rec.first + p) + (p == 0 ? 1 : 0)) * M + r;
    };
    float m = -FLT_MAX, l = 0.f, acc[W];
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {              // lane i: the weight of piece i0 + i
      const float z = i0 + lane < n ? sc.lse2[row_of(i0 + lane)] : -INFINITY;
      float nm = fmaxf(m, z);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, o));
      const float f = exp2_approx(m - nm), wz = z == -INFINITY ? 0.f : exp2_approx(z - nm);
      m = nm;
      l *= f;
#pragma unroll
      for (int e = 0; e < W; ++e) acc[e] *= f;
      const int k = min(32, n - i0);
#pragma unroll 8
      for (int i = 0; i < k; ++i) {
        const float wi = __shfl_sync(0xffffffffu, wz, i);
        const float2* src = reinterpret_cast<const float2*>(sc.o + row_of(i0 + i) * D) + lane;
        l += wi;
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {               // dims 64 e + 2 lane, + 1
          const float2 v = src[32 * e];
          acc[2 * e] = fmaf(wi, v.x, acc[2 * e]);
          acc[2 * e + 1] = fmaf(wi, v.y, acc[2 * e + 1]);
        }
      }
    }
    if (S > 1) {
      __syncthreads();                                // the unit before has been read
      if (sub > 0) {
#pragma unroll
        for (int e = 0; e < W / 2; ++e) part[warp][e][lane] = make_float2(acc[2 * e], acc[2 * e + 1]);
        if (lane == 0) ml[warp] = make_float2(m, l);
      }
      __syncthreads();
      for (int o = warp + 1; sub == 0 && o < warp + S; ++o) {
        const float2 z = ml[o];
        const float nm = fmaxf(m, z.x), f = exp2_approx(m - nm), fo = exp2_approx(z.x - nm);
        m = nm;
        l = fmaf(l, f, z.y * fo);
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
          const float2 v = part[o][e][lane];
          acc[2 * e] = fmaf(acc[2 * e], f, v.x * fo);
          acc[2 * e + 1] = fmaf(acc[2 * e + 1], f, v.y * fo);
        }
      }
    }
    if (sub > 0 || r >= it.rows) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t orow = it.q_row(a, (uint32_t)a.hq / (uint32_t)a.hk, it.row0 + r);
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D) + lane;
#pragma unroll
    for (int e = 0; e < W / 2; ++e) dst[32 * e] = X::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (a.lse && lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

// Whether pairs of CTAs take the batch (paged_prefill_pair.cu): head dim 256,
// pages that TMA can fetch, and sequences of more rows than a CTA's tile on average.
bool use_pair(const PagedAttnArgs& a, int head_dim) {
  return head_dim == 256 && paged_prefill_box(a.kv.page_size) > 1 && a.T * (a.hq / a.hk) >= PAIR_ROWS * a.B;
}

// Tile slots of the batch, and the CTAs (or pairs) that walk them.
int64_t slots_of(const PagedAttnArgs& a, int head_dim) {
  const int m = use_pair(a, head_dim) ? 256 : 128;
  return (a.T * (a.hq / a.hk) + m - 1) / m + a.B;
}
int walkers_of(const PagedAttnArgs& a, int head_dim, int num_sms) {
  const int most = num_sms < MAX_CTAS ? num_sms : MAX_CTAS;
  return use_pair(a, head_dim) ? most / 2 : most;
}
// Whether items may be cut over the CTAs: where one long sequence would keep a CTA
// busy long after the others (64 x 5 tokens over 2000 to 30000 keys: 609 us whole,
// 237 cut; 64 x 21: 574 and 340).  The kernel decides by the lengths; where whole items
// are quicker after all, it costs 3 to 8 us to find out (64 tokens over 300 keys:
// 14.4 us and 18; 16 x 100 over 1000: 66 and 74).  Two limits are the walk's, which
// counts one item a thread in a kernel that loads by TMA, and cost where lengths are
// mixed: 64 x 5 tokens over 2000 to 30000 keys with 32 + 8 heads of 128 are 592
// items, dealt out whole in 602 us, where 50 such sequences (482 items, 80 % of the
// keys) are cut and take 373; 37 tokens over 20011 keys take 400 to 414 us with pages
// of 1, 8 or 24 tokens, 41 with pages of 64.
bool may_cut(const PagedAttnArgs& a, int head_dim) {
  const int64_t items = slots_of(a, head_dim) * a.hk;
  return paged_prefill_box(a.kv.page_size) > 1 && items <= MAX_EVEN;
}

template <class E, int D, bool TMA, bool EVEN>
cudaError_t launch_attn(const Args& x, int grid, cudaStream_t s) {
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_done[dev]) {
    e = prepare_launch(paged_prefill_kernel<E, D, TMA, EVEN>, SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev] = true;
  }
  Args y = x;
  y.a.inject = take_debug_injection(QSA_INJECT_PAGED_STALL);
  paged_prefill_kernel<E, D, TMA, EVEN><<<grid, THREADS, SMEM, s>>>(y);
  return cudaGetLastError();
}

template <class E, int D, int M>
cudaError_t launch_join(const Args& x, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(JOIN_CTAS);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_prefill_join_kernel<E, D, M>, x);
}

template <class E, int D>
cudaError_t launch_d(const PagedAttnArgs& a, const CUtensorMap& tk, int num_sms, cudaStream_t s, bool join) {
  Args x;
  x.tk = tk;
  x.tv = tk;
  x.a = a;
  x.n_slots = slots_of(a, D);
  const int walkers = walkers_of(a, D, num_sms);
  x.box = paged_prefill_box(a.kv.page_size);
  if (join) {
    if constexpr (D == 256)
      if (use_pair(a, D)) return launch_join<E, D, 256>(x, s);
    return launch_join<E, D, 128>(x, s);
  }
  if (may_cut(a, D)) return launch_attn<E, D, true, true>(x, walkers, s);
  return x.box > 1 ? launch_attn<E, D, true, false>(x, walkers, s) : launch_attn<E, D, false, false>(x, walkers, s);
}

}  // namespace

size_t paged_prefill_scratch(int head_dim) { return REC_BYTES + (size_t)2 * MAX_CTAS * 128 * (head_dim + 1) * 4; }

bool paged_prefill_splits(const PagedAttnArgs& a, int head_dim) { return may_cut(a, head_dim); }

int paged_prefill_box(int page_size) {
  return page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : page_size % 16 == 0 ? 16 : 1;
}

cudaError_t launch_paged_prefill(const PagedAttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int head_dim,
                                 int dtype, int num_sms, cudaStream_t s, bool join) {
  if (a.B <= 0 || a.T <= 0) return cudaSuccess;
  if (!join && use_pair(a, head_dim)) {
    return launch_paged_prefill_pair(a, tk, tv, dtype, slots_of(a, head_dim), walkers_of(a, head_dim, num_sms),
                                     may_cut(a, head_dim), s);
  }
  const bool bf = dtype == QSA_DTYPE_BF16;
  switch (head_dim) {
    case 64: return bf ? launch_d<__nv_bfloat16, 64>(a, tk, num_sms, s, join)
                        : launch_d<__half, 64>(a, tk, num_sms, s, join);
    case 128: return bf ? launch_d<__nv_bfloat16, 128>(a, tk, num_sms, s, join)
                        : launch_d<__half, 128>(a, tk, num_sms, s, join);
    case 256: return bf ? launch_d<__nv_bfloat16, 256>(a, tk, num_sms, s, join)
                        : launch_d<__half, 256>(a, tk, num_sms, s, join);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qsa
