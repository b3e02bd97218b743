// What the two prefill kernels share: waits, TMA and tcgen05 instructions, the
// items of a ragged batch, and the softmax warps.
#pragma once
#include <cfloat>
#include <type_traits>

#include "paged.cuh"

namespace qsa {
namespace {

constexpr int KT = 128;                             // keys of a tile
constexpr int THREADS = 512;
constexpr int REGS_SOFT = 184, REGS_REST = 72;
static_assert(256 * (REGS_SOFT + REGS_REST) <= 65536, "register split");
constexpr int W_LOAD = 8, LWARPS = 4, W_MMA = 12, W_TMA = 13, W_PV = 14;   // warp 15 only makes up the warpgroup
constexpr int LOADERS = 32 * LWARPS;
constexpr int RT = LOADERS / 8, RJ = KT / RT;       // cp.async: rows of a pass, passes of a tile
// tiles whose row bits are live: K runs at most 6 tiles ahead of S (D = 64: the
// ring holds 5), S 2 ahead of the softmax
constexpr int NOK = 16;
constexpr uint32_t TMEM_COLS = 512;
// TMEM columns.  Where they suffice, P has two buffers (64 columns) apart from S
// (128), so that S is free as soon as its scores are in registers: with O of up to
// 128 columns S has two buffers, in a pair (256) one.  One CTA with 256 columns of
// O has two buffers in which P replaces the scores.
template <int D, bool PAIR>
struct Tmem {
  static constexpr bool APART = PAIR || D <= 128;
  static constexpr uint32_t O = D <= 128 ? 384 : 256;
  static __device__ __forceinline__ uint32_t s(uint32_t buf) { return PAIR ? 0 : 128 * buf; }
  static __device__ __forceinline__ uint32_t p(uint32_t buf) { return PAIR ? 128 + 64 * buf : APART ? 256 + 64 * buf : 128 * buf; }
};
constexpr int MAX_CTAS = 160;                       // bound of the scratch (148 SMs on B200)
constexpr int MAX_EVEN = THREADS;                   // most items that may be cut over the CTAs
// In tiles (of 1 to 2 us): what an item costs beside its own (its queries, the
// first scores, the last products and the results); the least that is worth a CTA;
// what the pieces and their join cost, with half of the walk for its second and
// third piece.  (37 tokens over 20K keys: whole 163 tiles in a row and 225 us, cut 8
// and 40 us; 5 over 1000: 14 and 23.5, 4 and 20.6 us; but 64 over 300: 9 and 18, 4
// and 21 us; 16 x 100 over 1000: 45 and 79, 32 and 81 us; 2000 over none: 48 and 72,
// 36 and 79 us.)
constexpr int ITEM_COST = 6, LEAST = 4, JOIN_COST = 7;
__host__ __device__ constexpr int64_t cut_cost(int64_t base) { return base + base / 2 + JOIN_COST; }
// setmaxnreg.inc takes from what the launch allotted: the kernel must have been
// compiled to the registers that the split adds up to, or it would wait for ever.
template <class F>
cudaError_t prepare_launch(F* kernel, uint32_t smem) {
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, kernel);
  if (e != cudaSuccess) return e;
  if (at.numRegs * THREADS < 256 * (REGS_SOFT + REGS_REST)) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}
// Quarter of a tile's exponentials after which the next tile's begin.  Builds in turn
// on one GPU, after quarter 1, 2 and 3: head dim 256 (24 + 2 heads) 4096 tokens 202,
// 200 and 190 us, 8 x 500 over 2000 227, 224 and 211, 16K and 32K tokens the same within
// 0.3 %; head dim 128 (32 + 8) 16K 2.20, 2.28 and 2.35 ms, 4096 tokens 172, 174 and
// 178 us; head dim 64 (16) 16K 904, 858 and 882 us, 4 x 4000 273, 261 and 266.
__host__ __device__ constexpr int turn_after(int D) { return D == 256 ? 3 : D == 128 ? 1 : 2; }
// Lazy maximum: a tile raises it when its own exceeds it by more than RAISE, and P is
// held times 2^P_SHIFT, so it stays below 2^(RAISE + P_SHIFT).  In fp16 (largest
// 2^16, normal numbers from 2^-14 on) the shift keeps the bits of weights down to
// 2^-21 of the maximum, and some down to 2^-32, where a first key outweighs the
// others; without it they would lose bits from 2^-14 on and vanish at 2^-25.  (16K
// tokens of 32 + 8 heads of 128 in fp16: 2.29 ms with and without the shift; a margin of
// 6 with a shift of 9 2.31, of 4 with 11 2.53: more rescaling.)
constexpr float RAISE = 8.f;
template <class E>
constexpr float P_SHIFT = std::is_same<E, __half>::value ? 7.f : 0.f;

__device__ __forceinline__ uint32_t swz128(uint32_t row, uint32_t c16) {
  return row * 128u + ((c16 ^ (row & 7u)) << 4);
}
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// mbar_wait that sees an abort at once.  CLUSTER: the arrivals may come from the
// other CTA of a pair.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t ok;
    if (CLUSTER)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
    else
      ok = mbar_try_wait(bar, parity);
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
// One arrival on the same barrier of the pair's first CTA.  MEMORY: it also
// releases this thread's shared-memory writes to the pair (a wait of about 1000
// cycles for all writes in flight); without, it orders what tcgen05 waits and
// fences have completed: accesses to TMEM.
template <bool MEMORY>
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(bar)));
  if (MEMORY) asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
  else asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
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
// GROUP 2: one MMA over the pair's two CTAs, issued by the first: each holds half
// of A's rows (and of D's) and half of B's columns, at the same addresses.
// D[tmem] (+)= A[smem] * B[smem]^T
template <int GROUP = 1>
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  if (GROUP == 1)
    asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
  else
    asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
template <int GROUP = 1>
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  if (GROUP == 1)
    asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
  else
    asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
template <int GROUP = 1>
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  if (GROUP == 1)
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar))
        : "memory");
  else   // on the same barrier of both CTAs
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
        ::"r"(smem_u32(bar)), "h"((uint16_t)3)
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

// What the join needs to know of an item: the CTAs (or pairs) that have its first
// and its last tile; last -1: one has it whole.
struct JoinRec { int32_t first, last; };
// A CTA has up to two pieces of shared items: 2c + 1 of one that starts with it, 2c
// of one that came in from before; 128 rows of D (a pair's 256) and their base-2
// log-sum-exp.
struct Scratch {
  JoinRec* rec;             // [MAX_EVEN]
  float* lse2;              // [2 MAX_CTAS][128]
  float* o;                 // [2 MAX_CTAS][128][D]
};
constexpr size_t REC_BYTES = 4096;
static_assert(MAX_EVEN * sizeof(JoinRec) <= REC_BYTES, "join records");
__host__ __device__ inline Scratch scratch_of(void* p) {
  uint8_t* u = static_cast<uint8_t*>(p);
  float* f = reinterpret_cast<float*>(u + REC_BYTES);
  return {reinterpret_cast<JoinRec*>(u), f, f + 2 * MAX_CTAS * 128};
}

struct Args {
  CUtensorMap tk, tv;       // pages, boxes of `box` rows x 64 dims (tv: the pair kernel's)
  PagedAttnArgs a;
  int64_t n_slots;          // tile slots of the batch
  int box;                  // 16, 32 or 64, or 1: no TMA
};

// Item w of M query rows.  Sequence b owns the tile slots from cu[b] per / M + b on (at least
// as many as it has tiles), so a slot's sequence is found by bisection and the
// slots without a tile are items without keys.  Rows (token, head) of the batch are
// below 2^30.
template <int M>
struct Item {
  int b, g, rows;           // sequence, KV head, rows in use
  int all, n_tiles, tile0;  // tiles; those of this CTA (n_tiles from tile0 on)
  int lo, ns, n_vis;        // key number v: v < ns ? v : lo + v - ns (whole boxes)
  int first, end;           // keys needed: [first, end) and those below the sinks
  int t0, row0;             // the sequence's first token row; first flat row of the item
  int64_t p0;               // position of the first row's token (of any length that the call was given)
  __device__ __forceinline__ Item(const Args& x, int64_t w) {
    const PagedAttnArgs& a = x.a;
    const uint32_t per = (uint32_t)a.hq / (uint32_t)a.hk;
    all = n_tiles = tile0 = 0;
    const int64_t turn = div64(w, a.hk);
    g = (int)(w - turn * a.hk);
    const int slot = (int)(x.n_slots - 1 - turn), T = (int)a.T;
    auto first_slot = [&](int seq, int row) { return first_tile_slot(seq, row, T, per, M); };
    int l = 0, h = a.B;
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (first_slot(mid, __ldg(a.cu_new + mid)) <= slot) l = mid; else h = mid;
    }
    b = l;
    t0 = __ldg(a.cu_new + b);
    const int t1 = min(__ldg(a.cu_new + b + 1), T);
    const int L = __ldg(a.cache_len + b);
    const int tile = slot - first_slot(b, t0);
    if (t0 < 0 || t0 >= t1 || tile < 0 || L < 0) return;
    const int n_rows = (t1 - t0) * (int)per;
    row0 = tile * M;
    rows = min(M, n_rows - row0);
    if (rows <= 0) return;
    const int64_t pos = (int64_t)L + (uint32_t)row0 / per, last = (int64_t)L + (uint32_t)(row0 + rows - 1) / per;
    end = (int)min(last + 1, (int64_t)a.kv.capacity);
    if (last >= a.kv.capacity) report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
    first = a.window > 0 && pos >= a.window ? (int)min(pos - a.window + 1, (int64_t)end) : 0;
    lo = first / x.box * x.box;
    ns = min((a.sinks + x.box - 1) / x.box * x.box, lo);
    if (ns == lo) ns = lo = 0;                      // no gap
    n_vis = ns + end - lo;
    p0 = pos;
    // at least one tile: rows whose keys all lie past the table come out zero
    n_tiles = all = max((n_vis + KT - 1) / KT, 1);
  }
  // Row of q and out of flat row f of the sequence.
  __device__ __forceinline__ int64_t q_row(const PagedAttnArgs& a, uint32_t per, uint32_t f) const {
    const uint32_t t = f / per;
    return (int64_t)(t0 + (int)t) * a.hq + (g * (int)per + (int)(f - t * per));
  }
  // only tiles [from, to)
  __device__ __forceinline__ void cut(int from, int to) {
    tile0 = from;
    n_tiles = min(all, to) - from;
  }
};

// The items of a CTA (or pair): w, w + step, .. last; of the first the tiles from
// `from` on, of the last those before `to`.
struct Walk {
  int w, last, step;
  int from, to;
};
// Number of an item: of up to MAX_EVEN that may be cut, or of any.
template <bool EVEN> using ItemNo = std::conditional_t<EVEN, int, int64_t>;
template <int M, bool EVEN>
__device__ __forceinline__ Item<M> item_of(const Args& x, const Walk& k, ItemNo<EVEN> w) {
  Item<M> it(x, w);
  if (EVEN && it.n_tiles > 0) it.cut(w == k.w ? k.from : 0, w == k.last ? k.to : INT32_MAX);
  return it;
}
// The same, through shuffles that tell the compiler that a warp has one walk.
__device__ __forceinline__ Walk uniform(const Walk& k) {
  auto one = [](auto v) { return __shfl_sync(0xffffffffu, v, 0); };
  return {one(k.w), one(k.last), one(k.step), one(k.from), one(k.to)};
}
// All threads of a CTA, once: the walk of CTA (or pair) c of n over up to MAX_EVEN
// items.  ITEM_COST units and a unit a tile for each, end to end, cut evenly, where
// that is quicker than whole items in turn (of those with tiles, if they are no more
// than two to a CTA, else of all).  Each thread counts one item's; those that hold
// the range's ends write them down.  buf: 3 KB of shared memory.
template <int M>
__device__ __forceinline__ Walk make_walk(const Args& x, int c, int n, void* buf) {
  const int n_items = (int)(x.n_slots * x.a.hk);
  int64_t* sum = static_cast<int64_t*>(buf);                        // [16]
  Walk* out = reinterpret_cast<Walk*>(sum + 16);
  int32_t* item = reinterpret_cast<int32_t*>(out + 1);              // [MAX_EVEN] the items with tiles
  int32_t* whole = item + MAX_EVEN;                                 // [MAX_CTAS] units of a CTA that takes whole items
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Scratch sc = scratch_of(x.a.scratch);
  const int tiles = tid < n_items ? Item<M>(x, tid).all : 0;
  const int64_t units = tiles ? tiles + ITEM_COST : 0;
  constexpr int64_t ONE = (int64_t)1 << 40;                         // sums: units, and above them items
  const int64_t mine = tiles ? ONE + units : 0;
  int64_t s = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += v;
  }
  if (lane == 31) sum[warp] = s;
  if (tid < MAX_CTAS) whole[tid] = 0;
  if (tid == 0) *out = {0, -1, 1, 0, 0};
  __syncthreads();
  int64_t total = 0, at = s - mine;                                 // at: before this item
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) at += sum[i];
    total += sum[i];
  }
  const int busy = (int)(total / ONE), rank = (int)(at / ONE);      // items with tiles; those before this one
  const bool two = busy <= 2 * n;
  total %= ONE;
  at %= ONE;
  if (tiles) {
    item[rank] = tid;
    atomicAdd(&whole[(two ? rank : tid) % n], (int)units);
  }
  __syncthreads();
  // CTAs beyond what is worth one have none
  const int64_t parts = min((int64_t)n, max(total / LEAST, (int64_t)1));
  const EvenCut range(total, parts);
  const bool cut = __syncthreads_or(tid < n && whole[tid] > cut_cost(range.base));
  if (c == 0 && tid < n_items && (!cut || !units)) sc.rec[tid] = {0, -1};
  if (!cut && !two) return {c, n_items - 1, n, 0, INT32_MAX};
  if (!cut) {
    if (c >= busy) return {0, -1, 1, 0, 0};
    const int w = item[c], last = c + n < busy ? item[c + n] : w;
    return {w, last, max(last - w, 1), 0, INT32_MAX};
  }
  if (c < parts && units) {
    const int64_t ua = range.begin(c), ub = range.begin(c + 1);
    const int64_t tile0 = at + ITEM_COST, end = tile0 + tiles;      // the item's tiles
    const int from = (int)max(ua - tile0, (int64_t)0), to = (int)max(min(ub, end) - tile0, (int64_t)0);
    if (at <= ua && ua < end) {
      out->w = tid;
      out->from = from;
    }
    if (at < ub && ub <= end) {
      out->last = tid;
      out->to = to;
    }
    if (ua <= tile0 && tile0 < ub) {                                // its first tile is here
      sc.rec[tid] = {c, to < tiles ? (int32_t)range.owner(end - 1) : -1};
    }
  }
  __syncthreads();
  return *out;
}

// The softmax warps (0-7): row r0 + r of an item of ROWS rows in TMEM lane r; cta:
// number of the CTA (or pair).  In a pair of CTAs (PAIR) the MMA's barriers are the first
// CTA's.
struct SoftBars {
  uint64_t *s_full, *s_empty, *p_full, *pv_done, *hand, *turn, *xbar, *o_empty;
};
template <class E, int D, int ROWS, bool PAIR, bool EVEN>
__device__ __forceinline__ void softmax_role(const Args& x, uint8_t* smem, uint32_t off_ok, uint32_t off_xch, const SoftBars& bar,
                                             uint32_t tmem, int warp, int lane, int r0, const Walk& walk, ItemNo<EVEN> w_first,
                                             ItemNo<EVEN> w_last, ItemNo<EVEN> w_step, int cta,
                                             volatile int* abort_flag) {
  using X = Elem<E>;
  using TM = Tmem<D, PAIR>;
  const PagedAttnArgs& a = x.a;
  const uint32_t per = (uint32_t)a.hq / (uint32_t)a.hk;
  const int quad = warp & 3, wg = warp >> 2;      // rows 32 quad .., tiles with count % 2 == wg
  const int r = 32 * quad + lane;
  const uint32_t lanes = (uint32_t)(32 * quad) << 16;
  volatile float* m_pub = reinterpret_cast<volatile float*>(smem + off_xch);      // [2][128]
  volatile float* l_pub = m_pub + 2 * 128;                                          // [2][128]
  uint32_t count = 0, items_done = 0;             // count: tiles of the items before
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, bar_wait<PAIR>(bar, parity, abort_flag, a.err));
  };
  for (ItemNo<EVEN> w = w_first; ok && w <= w_last; w += w_step) {
    int n_tiles, v0;                                // tiles of the item, first key number of the tile
    int v_min, v_max;                               // the row sees v in [v_min, v_max] and v < sinks
    int all_min, all_max;                           // every row sees v in [all_min, all_max]
    int64_t orow;                                   // output row, or piece row; -1: row not in use
    bool part;
    {
      const Item<ROWS> it = item_of<ROWS, EVEN>(x, walk, w);
      if (it.n_tiles <= 0) continue;
      n_tiles = it.n_tiles;
      v0 = it.tile0 * KT;
      const bool in = r0 + r < it.rows;
      const uint32_t flat = it.row0 + (in ? r0 + r : 0), row0 = it.row0, tok0 = row0 / per;
      const int shift = it.ns - it.lo;              // position -> number, behind the gap
      const int64_t pos = it.p0 + (int)(flat / per - tok0);
      const int64_t pos1 = it.p0 + (int)((row0 + min(it.rows, r0 + 128) - 1) / per - tok0);
      const int64_t pos_f = it.p0 + (int)((row0 + min(r0, it.rows - 1)) / per - tok0);
      v_max = (int)min(pos + shift, (int64_t)it.n_vis - 1);
      all_max = (int)min(pos_f + shift, (int64_t)it.n_vis - 1);
      // (numbers from n_vis on are none: a position may pass 2^31, a number may not)
      auto from = [&](int64_t p) { return a.window > 0 ? (int)min(max(p - a.window + 1 + shift, (int64_t)0), (int64_t)it.n_vis) : 0; };
      v_min = from(pos);
      all_min = from(pos1);
      part = EVEN && it.n_tiles < it.all;
      orow = !in ? -1 : part ? (int64_t)(2 * cta + (it.tile0 == 0 ? 1 : 0)) * ROWS + r0 + r : it.q_row(a, per, flat);
    }
    float m = -FLT_MAX, l = 0.f;
    for (int i = (int)((count ^ wg) & 1); i < n_tiles; i += 2) {
      const uint32_t n = count + i, buf = wg;     // n % 2 == wg
      if (!wait(&bar.s_full[buf], (n >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      const uint32_t s_addr = tmem + lanes + TM::s(buf), p_addr = tmem + lanes + TM::p(buf);
      float s[4][32];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(s_addr + 32 * q, s[q]);
      // the keys that are there, four to a byte
      const uint4* there = reinterpret_cast<const uint4*>(smem + off_ok + (n % NOK) * 32);
      const uint4 t0 = there[0], t1 = there[1];
      const int vt = v0 + i * KT;
      const bool whole = vt + KT - 1 <= all_max && (vt >= all_min || vt + KT <= a.sinks) &&
                         (t0.x & t0.y & t0.z & t0.w & t1.x & t1.y & t1.z & t1.w) == 0x0f0f0f0fu;
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld_wait(s[q]);
      if (TM::APART) {                            // a later S may overwrite these
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) arrive_leader<false>(bar.s_empty);
          else mbar_arrive(&bar.s_empty[buf]);
        }
      }
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
          if (__all_sync(0xffffffffu, mask == ~0u)) continue;       // most quarters of a border tile
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
        if (!wait(&bar.hand[(wg ^ 1) * 4 + quad], ((n - 1) >> 1) & 1)) { ok = false; break; }
      }
      if (i > 0) {
        const float mp = m_pub[(wg ^ 1) * 128 + r];
        l *= exp2_approx(m - mp);
        m = mp;
      }
      // The P V of two tiles before is done: its P may be overwritten (where P shares
      // the scores' columns, this tile's S came after that).  Waited for before the
      // hand-over, because the other group's waits for this barrier's next phase go
      // by parity: without it they could pass on the phase before and rescale, or
      // read, an O that products are still being added to.
      if (TM::APART && n >= 2 && !wait(&bar.pv_done[buf], ((n >> 1) - 1) & 1)) { ok = false; break; }
      const bool raise = mt > m + RAISE;
      const float m_old = m;
      if (raise) m = mt;
      m_pub[wg * 128 + r] = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.hand[wg * 4 + quad]);
      if (__any_sync(0xffffffffu, raise)) {
        const float f = exp2_approx(m_old - m);
        l *= f;
        if (i > 0) {
          // O holds the tiles up to i - 1 once their P V is done; this tile's
          // waits for this warp
          if (!wait(&bar.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t o[16];
            const uint32_t ad = tmem + lanes + TM::O + 16 * cc;
            tmem_ld16(ad, o);                     // waits for the load
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(ad, o);
          }
        }
      }
      // The exponentials of a tile begin when those of the tile before are nearly
      // done.  The two warps of a scheduler share its special-function unit: side
      // by side they would take twice as long and leave it idle afterwards.
      if (n > 0 && !wait(&bar.turn[(wg ^ 1) * 4 + quad], ((n - 1) >> 1) & 1)) { ok = false; break; }
      // p = 2^(s scale - m + P_SHIFT); the sum takes the fp32 values, the products p
      // rounded to 16 bits
      const uint64_t sc2 = pk2(a.scale_log2, a.scale_log2), nm2 = pk2(P_SHIFT<E> - m, P_SHIFT<E> - m);
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
        tmem_st16(p_addr + 16 * q, pk);
        if (q == turn_after(D)) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.turn[wg * 4 + quad]);
        }
      }
      float l0, l1;
      upk2(sum, l0, l1);
      l += l0 + l1;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) arrive_leader<false>(&bar.p_full[buf]);
        else mbar_arrive(&bar.p_full[buf]);
      }
    }
    if (!ok) break;
    // ---- O / l
    count += n_tiles;
    const uint32_t n = count - 1;                 // the item's last tile
    if ((n & 1) != (uint32_t)wg) {                // the other group's: its maximum is the last
      if (!wait(&bar.hand[(wg ^ 1) * 4 + quad], (n >> 1) & 1)) { ok = false; break; }
      const float mp = m_pub[(wg ^ 1) * 128 + r];
      l *= exp2_approx(m - mp);
      m = mp;
    }
    // (this P V began after both groups had taken the item before's sums)
    if (!wait(&bar.pv_done[n & 1], (n >> 1) & 1)) { ok = false; break; }
    tc_fence_after();
    l_pub[wg * 128 + r] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.xbar[quad]);
    if (!wait(&bar.xbar[quad], items_done & 1)) { ok = false; break; }
    const float l_other = l_pub[(wg ^ 1) * 128 + r];
    const float lr = l + l_other;
    const float inv = lr == 0.f ? 0.f : 1.f / lr;   // no key at all: zero
    const float lse2 = lr == 0.f ? -INFINITY : m + log2f(lr) - P_SHIFT<E>;
    const Scratch sc = scratch_of(a.scratch);
    float ov[D / 64][32];                            // all loads at once
#pragma unroll
    for (int cc = 0; cc < D / 64; ++cc) tmem_ld32(tmem + lanes + TM::O + (D / 2) * wg + 32 * cc, ov[cc]);
#pragma unroll
    for (int cc = 0; cc < D / 64; ++cc) {
      float (&o)[32] = ov[cc];
      const int d0 = (D / 2) * wg + 32 * cc;
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
    if (lane == 0) {
      if (PAIR) arrive_leader<false>(bar.o_empty);
      else mbar_arrive(bar.o_empty);
    }
    ++items_done;
  }
}

}  // namespace
}  // namespace qsa
