// Attention of a ragged batch of new tokens over their pages (qsa_paged_prefill)
// on the 5th-generation tensor cores.
//
//   out[t][h] = sum_j softmax_j(q[t][h] . k[j] scale) v[j]
//
// over the keys j up to the token's own that window and sinks leave; one pass
// with a running maximum and sum.
//
// Item = (128 query rows of one sequence, KV head, range of keys); the rows are
// the sequence's (token, query head of the KV head) pairs laid out flat, so any
// head count fills the tiles and the heads of a KV head share its loads.  The
// keys that any row sees are numbered without the gap between sinks and window
// and taken in tiles of 128.  Persistent CTAs (one per SM) walk the items, those
// of the last tokens (the most keys) first.
//   * warps 0-7 (softmax): two warpgroups that take the tiles in turn, a thread a
//     query row (TMEM lane): mask, tile maximum, the running maximum from the
//     other group (raised only when a tile exceeds it by more than 8, so the
//     rescale of O is rare), handed back at once, then exp2 in base 2 and P
//     packed to 16 bits into the score buffer.  So one group's exponentials run
//     beside the other's loads and maxima.  At the end O / l and the log-sum-exp.
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
// Registers: 168 a softmax thread, 88 the others (setmaxnreg).
// Every mbarrier wait is bounded (timeout -> error word, clean exit): on an abort
// every role leaves its loop, the loaders wait for their own copies and the MMA
// thread for its last commit before TMEM is released.
//
// With few rows (a short chunk over a long prefix) an item's keys are cut into
// n_split ranges so that the SMs fill up; the ranges' results go to the scratch
// as normalised fp32 rows with their log-sum-exp, and the join kernel adds them
// in the order of the keys.
#include <cfloat>
#include <type_traits>

#include "paged.cuh"

namespace qsa {
namespace {

constexpr int KT = 128;                             // keys of a tile
constexpr int M = 128;                              // query rows of an item
constexpr int W_LOAD = 8, LWARPS = 4, W_MMA = 12, W_TMA = 13, W_PV = 14;
constexpr int LOADERS = 32 * LWARPS;
constexpr int THREADS = 512;                        // warp 15 only makes up the last warpgroup
constexpr int REGS_SOFT = 168, REGS_REST = 88;
static_assert(256 * (REGS_SOFT + REGS_REST) <= 65536, "register split");
constexpr int RT = LOADERS / 8, RJ = KT / RT;       // cp.async: rows of a pass, passes of a tile
constexpr uint32_t SLOT = 16384;
constexpr int NS = 5;                               // slots of the K ring and of the V ring
constexpr uint32_t OFF_K = 65536;                   // Q: up to 128 rows x 512 B
constexpr uint32_t OFF_V = OFF_K + NS * SLOT;
constexpr uint32_t OFF_XCH = OFF_V + NS * SLOT;     // running maxima [2][128], row sums [2][128]
constexpr uint32_t OFF_OK = OFF_XCH + 2048;         // rows that are there, of NOK tiles, 32 bytes each
// tiles whose row bits are live: K runs at most 6 tiles ahead of S (D = 64: the
// ring holds 5), S 2 ahead of the softmax
constexpr int NOK = 16;
constexpr uint32_t OFF_BAR = OFF_OK + 32 * NOK;
constexpr uint32_t SMEM = OFF_BAR + 384;
static_assert(SMEM <= 232448, "prefill smem");
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_S = 0, TM_O = 256;            // S / P buffers at 0 and 128
constexpr int MAX_PIECES = 160;                     // bound of the scratch
constexpr int MAX_SPLIT = 32;
constexpr float RAISE = 8.f;                        // lazy maximum: P stays below 2^8

__device__ __forceinline__ uint32_t swz128(uint32_t row, uint32_t c16) {
  return row * 128u + ((c16 ^ (row & 7u)) << 4);
}
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// mbar_wait with the thread suspended for up to 10 us at a time instead of
// polling: sixteen warps that poll slow the others' shared-memory and
// special-function instructions.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(10000u)
        : "memory");
    if (ok) return true;
    if (it == 0) t0 = globaltimer();
    if (*abort_flag) return false;
    if (globaltimer() - t0 > QSA_WAIT_TIMEOUT_NS) {
      *abort_flag = 1;
      report_error(err, QSA_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
}
// The barrier's phase waits for this thread's copies so far, beside its counted
// arrivals (this form adds the arrival that it makes to the pending count).
__device__ __forceinline__ void cp_async_hold(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// A box of a page: dims, rows of the page, KV head, page (no multicast).
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* m, int32_t dim, int32_t row, int32_t head,
                                             int32_t page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(dim), "r"(row), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}
// Operand descriptors, 128-byte swizzle, as constant fields and a start address:
// K-major (rows of 64 elements, 8-row groups 1024 bytes apart) and MN-major (lbo
// bytes between 64-element atoms along N, 1024 between 8-row groups along K).
constexpr uint64_t DESC_K = (uint64_t)1u << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1u << 46 | (uint64_t)2u << 61;
__host__ __device__ constexpr uint64_t desc_mn(uint32_t lbo) {
  return (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
__device__ __forceinline__ uint64_t desc_at(uint64_t fields, uint32_t addr) { return fields | (addr >> 4); }
// The MMA warp stays converged and one elected lane issues (always the same one):
// descriptors and addresses then live in uniform registers.  Inside a one-lane
// branch each MMA first moves them there, which took longer than the MMA.
// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

struct Grid {
  int64_t n_slots;          // tile slots of the batch
  int n_split;
};
struct Scratch {
  float* lse2;              // [MAX_PIECES][128]
  float* o;                 // [MAX_PIECES][128][D]
};
__host__ __device__ inline Scratch scratch_of(void* p) {
  return {static_cast<float*>(p), static_cast<float*>(p) + MAX_PIECES * M};
}

struct Args {
  CUtensorMap tk;           // K pages, boxes of `box` rows x 64 dims
  PagedAttnArgs a;
  Grid grid;
  int box;                  // 16, 32 or 64, or 1: no TMA
};

// Item w.  Sequence b owns the tile slots from cu[b] per / 128 + b on (at least
// as many as it has tiles), so a slot's sequence is found by bisection and the
// slots without a tile are items without keys.
struct Item {
  int b, g, rows;           // sequence, KV head, rows in use
  int n_tiles, tile0;       // tiles of this range, its first
  int pieces, split;        // ranges that the item's keys are cut into, which one this is
  int lo, ns, n_vis;        // key number v: v < ns ? v : lo + v - ns (whole boxes)
  int first, end;           // keys needed: [first, end) and those below the sinks
  int p0;                   // position of the first row's token
  int64_t t0, row0;         // the sequence's first token row; first flat row of the item
  __device__ __forceinline__ Item(const Args& x, int64_t w) {
    const PagedAttnArgs& a = x.a;
    const int per = a.hq / a.hk, ns_ = x.grid.n_split;
    n_tiles = 0;
    tile0 = 0;
    split = (int)(w % ns_);
    w /= ns_;
    g = (int)(w % a.hk);
    const int64_t slot = x.grid.n_slots - 1 - w / a.hk;
    int l = 0, h = a.B;
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if ((int64_t)__ldg(a.cu_new + mid) * per / M + mid <= slot) l = mid; else h = mid;
    }
    b = l;
    t0 = __ldg(a.cu_new + b);
    const int64_t t1 = min((int64_t)__ldg(a.cu_new + b + 1), a.T);
    const int L = __ldg(a.cache_len + b);
    const int64_t tile = slot - (t0 * per / M + b), n_rows = (t1 - t0) * per;
    row0 = tile * M;
    rows = (int)min((int64_t)M, n_rows - row0);
    if (t0 < 0 || tile < 0 || rows <= 0 || L < 0) return;
    const int64_t pos = L + row0 / per, last = L + (row0 + rows - 1) / per;
    end = (int)min(last + 1, (int64_t)a.kv.capacity);
    if (last >= a.kv.capacity) report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
    first = a.window > 0 && pos >= a.window ? (int)min(pos - a.window + 1, (int64_t)end) : 0;
    lo = first / x.box * x.box;
    ns = min((a.sinks + x.box - 1) / x.box * x.box, lo);
    if (ns == lo) ns = lo = 0;                      // no gap
    n_vis = ns + end - lo;
    p0 = (int)min(pos, (int64_t)INT32_MAX);
    // at least one tile: rows whose keys all lie past the table come out zero
    const int all = max((n_vis + KT - 1) / KT, 1), each = (all + ns_ - 1) / ns_;
    pieces = (all + each - 1) / each;
    tile0 = split * each;
    n_tiles = min(each, all - tile0);
  }
};

template <class E, int D, bool TMA>
__global__ void __launch_bounds__(THREADS, 1) paged_prefill_kernel(const __grid_constant__ Args x) {
  constexpr int NCH = D / 64;                       // 64-dim chunks: K (and V) slots of a tile
  constexpr int KV = KT / NCH;                      // keys of a V slot
  constexpr int GR = NCH < 2 ? 1 : 2;               // slots to a "full" barrier
  constexpr uint32_t IDESC = umma_idesc_bf16_f32(M, KT) &
                             (std::is_same<E, __half>::value ? ~((1u << 7) | (1u << 10)) : ~0u);   // f16: 0
  constexpr uint32_t IDESC_PV = ((IDESC & ~(63u << 17)) | ((uint32_t)(D >> 3) << 17)) | (1u << 16);   // V MN-major
  using X = Elem<E>;
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
  uint64_t* p_full = s_full + 2;                    // [2]
  uint64_t* pv_done = p_full + 2;                   // [2]
  uint64_t* o_empty = pv_done + 2;
  uint64_t* hand = o_empty + 1;                     // [2][4]: the maximum after a tile, 32 rows each
  uint64_t* xbar = hand + 8;                        // [4]: row sums, 32 rows each
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
    for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 4); mbar_init(&pv_done[i], 1); }
    for (int i = 0; i < 8; ++i) mbar_init(&hand[i], 1);
    mbar_init(o_empty, 8);
    for (int i = 0; i < 4; ++i) mbar_init(&xbar[i], 2);
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) { tmem_alloc(tmem_slot, TMEM_COLS); tmem_relinquish(); }
  pdl_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t n_items = x.grid.n_slots * a.hk * x.grid.n_split;
  const int per = a.hq / a.hk;

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
    for (int64_t w = blockIdx.x; ok && w < n_items; w += gridDim.x) {
      const Item it(x, w);
      if (it.n_tiles <= 0) continue;
      const int32_t* table = a.kv.table + (int64_t)it.b * a.kv.table_ld;
      const int64_t head = (int64_t)it.g * a.kv.head_stride + 8 * c;
      auto key_of = [&](int v) { return v < it.ns ? v : it.lo + (v - it.ns); };
      // Page ids of this thread's rows rt + RT j of a tile: loaded a tile ahead,
      // all at once.
      int ids[RJ];
      auto load_ids = [&](int tile) {
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          const int key = key_of(max(min(tile * KT + RT * j + rt, it.n_vis - 1), 0));
          ids[j] = __ldg(table + page_of(a.kv, (uint32_t)min(key, a.kv.capacity - 1)));
        }
      };
      // A tile's rows: offset of this thread's chunk, and whether the row is there
      // (some query sees it and its page is one).
      struct Rows { int64_t off[RJ]; uint32_t ok; };
      auto find_rows = [&](int tile, Rows& d) {
        d.ok = 0;
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          const int v = tile * KT + RT * j + rt, key = key_of(v);
          const bool needed = v < it.n_vis && (key >= it.first || key < a.sinks);
          const bool good = needed && (uint32_t)ids[j] < (uint32_t)a.kv.n_pages;
          const int in_page = key - (int)(page_of(a.kv, (uint32_t)key) * (uint32_t)a.kv.page_size);
          d.off[j] = good ? (int64_t)ids[j] * a.kv.page_stride + (int64_t)in_page * a.kv.token_stride + head : 0;
          d.ok |= (uint32_t)good << j;
          bad |= (uint32_t)(needed && !good);
        }
        if (bad) report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
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
          const int64_t f = it.row0 + (valid ? r : 0);
          const uint16_t* src = a.q + ((it.t0 + f / per) * a.hq + it.g * per + f % per) * D + 8 * c;
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
    for (int64_t w = blockIdx.x; ok && w < n_items; w += gridDim.x) {
      const Item it(x, w);
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
    for (int64_t w = blockIdx.x; ok && w < n_items; w += gridDim.x) {
      const Item it(x, w);
      const int n_tiles = __shfl_sync(0xffffffffu, it.n_tiles, 0);
      if (n_tiles <= 0) continue;
      if (!wait(q_full, items_done & 1)) { ok = false; break; }
      fence_async_proxy();                          // Q: written by cp.async, read by the MMA
      for (int i = 0; i < n_tiles; ++i, ++count) {
        // S overwrites the buffer of the P two tiles before: its P V is done.
        // (That barrier's next phase needs this S, so its parity is exact.)
        if (count >= 2 && !wait(&pv_done[count & 1], ((count >> 1) - 1) & 1)) { ok = false; break; }
        const uint32_t d = tm + TM_S + 128 * (count & 1);
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
    for (int64_t w = blockIdx.x; ok && w < n_items; w += gridDim.x) {
      const Item it(x, w);
      const int n_tiles = __shfl_sync(0xffffffffu, it.n_tiles, 0);
      if (n_tiles <= 0) continue;
      if (items_done > 0 && !wait(o_empty, (items_done - 1) & 1)) { ok = false; break; }
      for (int i = 0; i < n_tiles; ++i, ++count) {
        const uint32_t p = tm + TM_S + 128 * (count & 1);
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
            umma_ts(tm + TM_O, p + 8 * (s * (KV / 16) + ks), desc_at(desc_mn(KV * 128), vb + 2048 * ks), IDESC_PV,
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
    const int quad = warp & 3, wg = warp >> 2;      // rows 32 quad .., tiles with count % 2 == wg
    const int r = 32 * quad + lane;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    volatile float* m_pub = reinterpret_cast<volatile float*>(smem + OFF_XCH);      // [2][128]
    volatile float* l_pub = m_pub + 2 * M;                                          // [2][128]
    uint32_t count = 0, items_done = 0;             // count: tiles of the items before
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, bar_wait(bar, parity, abort_flag, a.err));
    };
    for (int64_t w = blockIdx.x; ok && w < n_items; w += gridDim.x) {
      int n_tiles, v0;                                // tiles of the item, first key number of the tile
      int v_min, v_max;                               // the row sees v in [v_min, v_max] and v < sinks
      int all_min, all_max;                           // every row sees v in [all_min, all_max]
      int64_t orow;                                   // output row, or piece row; -1: row not in use
      bool part;
      {
        const Item it(x, w);
        if (it.n_tiles <= 0) continue;
        n_tiles = it.n_tiles;
        v0 = it.tile0 * KT;
        const bool in = r < it.rows;
        const int64_t flat = it.row0 + (in ? r : 0), tok0 = it.row0 / per;
        const int shift = it.ns - it.lo;              // position -> number, behind the gap
        const int64_t pos = (int64_t)it.p0 + (flat / per - tok0);
        const int64_t pos1 = (int64_t)it.p0 + ((it.row0 + it.rows - 1) / per - tok0);
        v_max = (int)min(pos + shift, (int64_t)it.n_vis - 1);
        all_max = (int)min((int64_t)it.p0 + shift, (int64_t)it.n_vis - 1);
        v_min = a.window > 0 ? (int)max(pos - a.window + 1 + shift, (int64_t)0) : 0;
        all_min = a.window > 0 ? (int)max(pos1 - a.window + 1 + shift, (int64_t)0) : 0;
        part = it.pieces > 1;
        orow = !in ? -1 : part ? w * M + r : (it.t0 + flat / per) * a.hq + it.g * per + flat % per;
      }
      float m = -FLT_MAX, l = 0.f;
      for (int i = (int)((count ^ wg) & 1); i < n_tiles; i += 2) {
        const uint32_t n = count + i, buf = wg;     // n % 2 == wg
        if (!wait(&s_full[buf], (n >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t s_addr = tmem + lanes + TM_S + 128 * buf;
        float s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(s_addr + 32 * q, s[q]);
        // the keys that are there, four to a byte
        const uint4* there = reinterpret_cast<const uint4*>(smem + OFF_OK + (n % NOK) * 32);
        const uint4 t0 = there[0], t1 = there[1];
        const int vt = v0 + i * KT;
        const bool whole = vt + KT - 1 <= all_max && (vt >= all_min || vt + KT <= a.sinks) &&
                           (t0.x & t0.y & t0.z & t0.w & t1.x & t1.y & t1.z & t1.w) == 0x0f0f0f0fu;
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_wait(s[q]);
        if (!whole) {
          const uint32_t bits[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
          auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
          auto squeeze = [](uint32_t x) -> uint32_t {   // four bits of each byte to 16
            x = (x | x >> 4) & 0x00ff00ffu;
            return (x | x >> 8) & 0xffffu;
          };
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int vq = vt + 32 * q;
            const uint32_t mask = (squeeze(bits[2 * q]) | squeeze(bits[2 * q + 1]) << 16) & below(v_max + 1 - vq) &
                                  (~below(v_min - vq) | below(a.sinks - vq));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(mask >> e & 1)) s[q][e] = -INFINITY;
          }
        }
        float mt = -INFINITY, mu = -INFINITY;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          mt = max3f(mt, s[0][e], s[1][e]);
          mu = max3f(mu, s[2][e], s[3][e]);
        }
        mt = fmaxf(fmaxf(mt, mu) * a.scale_log2, -FLT_MAX);   // a tile without a key leaves the maximum as it is
        // the maximum after the tile before, from the other group (also between
        // items, where it is not used, so that no barrier runs two phases ahead)
        if (n > 0) {
          if (!wait(&hand[(wg ^ 1) * 4 + quad], ((n - 1) >> 1) & 1)) { ok = false; break; }
        }
        if (i > 0) {
          const float mp = m_pub[(wg ^ 1) * M + r];
          l *= exp2_approx(m - mp);
          m = mp;
        }
        const bool raise = mt > m + RAISE;
        const float m_old = m;
        if (raise) m = mt;
        m_pub[wg * M + r] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&hand[wg * 4 + quad]);
        if (__any_sync(0xffffffffu, raise)) {
          const float f = exp2_approx(m_old - m);
          l *= f;
          if (i > 0) {
            // O holds the tiles up to i - 1 once their P V is done; this tile's
            // waits for this warp
            if (!wait(&pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < D / 16; ++cc) {
              uint32_t o[16];
              const uint32_t ad = tmem + lanes + TM_O + 16 * cc;
              tmem_ld16(ad, o);                     // waits for the load
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(ad, o);
            }
          }
        }
        // p = 2^(s scale - m); the sum takes the fp32 values, the products p
        // rounded to 16 bits.  P takes the first half of the scores' columns.
        const uint64_t sc2 = pk2(a.scale_log2, a.scale_log2), nm2 = pk2(-m, -m);
        uint64_t sum = pk2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0, x1;
            upk2(fma2(pk2(s[q][2 * e], s[q][2 * e + 1]), sc2, nm2), x0, x1);
            x0 = exp2_approx(x0);
            x1 = exp2_approx(x1);
            sum = add2(sum, pk2(x0, x1));
            pk[e] = X::pack(x0, x1);
          }
          tmem_st16(s_addr + 16 * q, pk);
        }
        float l0, l1;
        upk2(sum, l0, l1);
        l += l0 + l1;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      if (!ok) break;
      // ---- O / l
      count += n_tiles;
      const uint32_t n = count - 1;                 // the item's last tile
      if ((n & 1) != (uint32_t)wg) {                // the other group's: its maximum is the last
        if (!wait(&hand[(wg ^ 1) * 4 + quad], (n >> 1) & 1)) { ok = false; break; }
        const float mp = m_pub[(wg ^ 1) * M + r];
        l *= exp2_approx(m - mp);
        m = mp;
      }
      // (this P V began after both groups had taken the item before's sums)
      if (!wait(&pv_done[n & 1], (n >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      l_pub[wg * M + r] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&xbar[quad]);
      if (!wait(&xbar[quad], items_done & 1)) { ok = false; break; }
      const float l_other = l_pub[(wg ^ 1) * M + r];
      const float lr = l + l_other;
      const float inv = lr == 0.f ? 0.f : 1.f / lr;   // no key at all: zero
      const float lse2 = lr == 0.f ? -INFINITY : m + log2f(lr);
      const Scratch sc = scratch_of(a.scratch);
#pragma unroll 1
      for (int cc = 0; cc < D / 64; ++cc) {
        float o[32];
        const int d0 = (D / 2) * wg + 32 * cc;
        tmem_ld32(tmem + lanes + TM_O + d0, o);
        tmem_ld_wait(o);
        if (orow >= 0 && part) {
          float4* dst = reinterpret_cast<float4*>(sc.o + orow * D + d0);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q] = make_float4(o[4 * q] * inv, o[4 * q + 1] * inv, o[4 * q + 2] * inv, o[4 * q + 3] * inv);
        } else if (orow >= 0) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + orow * D + d0);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            dst[q] = make_uint4(X::pack(o[8 * q] * inv, o[8 * q + 1] * inv), X::pack(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                                X::pack(o[8 * q + 4] * inv, o[8 * q + 5] * inv),
                                X::pack(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
        }
      }
      if (orow >= 0 && wg == 0) {
        if (part) sc.lse2[orow] = lse2;
        else if (a.lse) a.lse[orow] = lse2 * 0.69314718055994531f;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
      ++items_done;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the ranges of items whose keys were cut: one warp a query row.
template <class E, int D>
__global__ void __launch_bounds__(256) paged_prefill_join_kernel(const __grid_constant__ Args x) {
  constexpr int W = D / 32;                         // dims of a lane: 2, 4 or 8
  using X = Elem<E>;
  const PagedAttnArgs& a = x.a;
  pdl_wait();
  const int64_t id = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5));
  const int64_t w0 = id / M * x.grid.n_split;       // the item's first range
  const int r = (int)(id % M), lane = threadIdx.x & 31;
  if (w0 >= x.grid.n_slots * a.hk * x.grid.n_split) return;
  const Item it(x, w0);
  if (it.n_tiles <= 0 || it.pieces <= 1 || r >= it.rows) return;
  const Scratch sc = scratch_of(a.scratch);
  float m = -FLT_MAX, l = 0.f, acc[W];
#pragma unroll
  for (int e = 0; e < W; ++e) acc[e] = 0.f;
  for (int i = 0; i < it.pieces; ++i) {
    const int64_t row = (w0 + i) * M + r;
    const float z = sc.lse2[row];
    float v[W];
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = sc.o[row * D + W * lane + e];
    if (z == -INFINITY) continue;                   // a range without a key
    const float nm = fmaxf(m, z), f0 = exp2_approx(m - nm), f1 = exp2_approx(z - nm);
    l = fmaf(l, f0, f1);
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] = fmaf(acc[e], f0, v[e] * f1);
    m = nm;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int per = a.hq / a.hk;
  const int64_t flat = it.row0 + r, orow = (it.t0 + flat / per) * a.hq + it.g * per + flat % per;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + W * lane);
#pragma unroll
  for (int e = 0; e < W / 2; ++e) dst[e] = X::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (a.lse && lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

Grid grid_of(const PagedAttnArgs& a, int num_sms) {
  Grid g;
  g.n_slots = (a.T * (a.hq / a.hk) + M - 1) / M + a.B;
  // ranges: as many as fill the SMs, from the slots (a sequence's last slot is
  // often empty, so the SMs are filled to about a half at the least)
  const int64_t n = (num_sms < MAX_PIECES ? num_sms : MAX_PIECES) / (g.n_slots * a.hk);
  g.n_split = (int)(n < 1 ? 1 : (n > MAX_SPLIT ? MAX_SPLIT : n));
  return g;
}

template <class E, int D, bool TMA>
cudaError_t launch_attn(const Args& x, int grid, cudaStream_t s) {
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(paged_prefill_kernel<E, D, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev] = true;
  }
  paged_prefill_kernel<E, D, TMA><<<grid, THREADS, SMEM, s>>>(x);
  return cudaGetLastError();
}

template <class E, int D>
cudaError_t launch_d(const PagedAttnArgs& a, const CUtensorMap& tk, int num_sms, cudaStream_t s, bool join) {
  Args x;
  x.tk = tk;
  x.a = a;
  x.grid = grid_of(a, num_sms);
  x.box = paged_prefill_box(a.kv.page_size);
  const int64_t items = x.grid.n_slots * a.hk * x.grid.n_split;
  if (!join) {
    const int grid = (int)(items < num_sms ? items : num_sms);
    return x.box > 1 ? launch_attn<E, D, true>(x, grid, s) : launch_attn<E, D, false>(x, grid, s);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items / x.grid.n_split * (M / 8)));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_prefill_join_kernel<E, D>, x);
}

}  // namespace

size_t paged_prefill_scratch(int head_dim) { return (size_t)MAX_PIECES * M * (head_dim + 1) * 4; }

bool paged_prefill_splits(const PagedAttnArgs& a, int num_sms) { return grid_of(a, num_sms).n_split > 1; }

int paged_prefill_box(int page_size) {
  return page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : page_size % 16 == 0 ? 16 : 1;
}

cudaError_t launch_paged_prefill(const PagedAttnArgs& a, const CUtensorMap& tk, int head_dim, int dtype, int num_sms, cudaStream_t s, bool join) {
  if (a.B <= 0 || a.T <= 0) return cudaSuccess;
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
