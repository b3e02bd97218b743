// Attention of a ragged batch of new tokens over their pages (qsa_paged_prefill)
// for head dim 256 and sequences of more than 128 query rows: one MMA over two CTAs.
//
// The mathematics, the numbering of the keys and the softmax are those of
// paged_prefill.cu.  There one CTA's tile of 128 rows needs 128 KB of K and V per
// 128 keys and 2060 cycles of MMA, more than its loads and its 227 KB of shared
// memory keep up with (Q alone is 64 KB).  Here a cluster of two CTAs takes 256
// rows: tcgen05 cta_group::2 with M = 256, each CTA with its 128 rows of Q, S, P
// and O and half of every operand B: 64 of a tile's 128 keys of K, 128 of the 256
// dims of V.  So each loads and holds half as much for the same products, two K
// tiles and three V tiles fit, all by TMA.
//   * warps 0-7 of both CTAs: softmax (paged_prefill.cuh); warps 8-11: Q; warp 13:
//     K and V halves by TMA, a box of 16 to 64 rows x 64 dims at a time.
//   * warp 12: S, warp 14: P V, both issued by the first CTA.  In the second one
//     the same warps tell the first that its halves have landed.  V rows that no
//     query sees, whose memory may hold anything, are set to zero before that.
//   * commits arrive on the barriers of both CTAs; the softmax warps of both
//     arrive on the first one's.
// Every wait is bounded, as there; the CTAs leave together.
// Bound by the tensor cores (a tile's products take 2060 cycles) and, over
// milliseconds, by the power limit: 32768 tokens of 24 + 2 heads of 256 take 9.4
// to 9.9 ms, 1330 to 1400 TFLOP/s by the clock that is left; 16384 tokens 2.2 to 2.5 ms
// with the tensor pipe 77 % busy; 8 sequences of up to 8192 with a window of 1024
// keys 0.57 to 0.68 ms in a replayed graph, 0.66 as single calls on fresh inputs, 840
// TFLOP/s of visible pairs (the tiles at both ends of a window are half masked).
#include "paged_prefill.cuh"

namespace qsa {
namespace {

constexpr int D = 256, M = 256;
constexpr uint32_t STAGE = 32768;                   // half a K tile: 64 keys x 256 dims; half a V tile: 128 x 128
constexpr int NK = 2, NV = 3;
constexpr uint32_t OFF_K = 65536;                   // Q: 128 rows x 512 B, chunks of 64 dims
constexpr uint32_t OFF_V = OFF_K + NK * STAGE;
constexpr uint32_t OFF_XCH = OFF_V + NV * STAGE;
constexpr uint32_t OFF_OK = OFF_XCH + 2048;
constexpr uint32_t OFF_BAR = OFF_OK + 32 * NOK;
constexpr uint32_t SMEM = OFF_BAR + 448;
static_assert(SMEM <= 232448, "prefill smem");

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <class E, bool EVEN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) paged_prefill_pair_kernel(const __grid_constant__ Args x) {
  constexpr uint32_t IDESC = umma_idesc_bf16_f32(M, KT) &
                             (std::is_same<E, __half>::value ? ~((1u << 7) | (1u << 10)) : ~0u);   // f16: 0
  constexpr uint32_t IDESC_PV = ((IDESC & ~(63u << 17)) | ((uint32_t)(D >> 3) << 17)) | (1u << 16);   // V MN-major
  using TM = Tmem<D, true>;
  const PagedAttnArgs& a = x.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);   // [NK] this CTA's half
  uint64_t* k_empty = k_full + NK;                  // [NK]
  uint64_t* v_full = k_empty + NK;                  // [NV]
  uint64_t* v_empty = v_full + NV;                  // [NV]
  uint64_t* k_peer = v_empty + NV;                  // [NK] the second CTA's half, in the first
  uint64_t* v_peer = k_peer + NK;                   // [NV]
  uint64_t* q_full = v_peer + NV;
  uint64_t* q_peer = q_full + 1;
  uint64_t* q_empty = q_peer + 1;
  uint64_t* s_full = q_empty + 1;                   // [2]
  uint64_t* s_empty = s_full + 2;
  uint64_t* p_full = s_empty + 1;                   // [2]
  uint64_t* pv_done = p_full + 2;                   // [2]
  uint64_t* o_empty = pv_done + 2;
  uint64_t* hand = o_empty + 1;                     // [2][4]
  uint64_t* turn = hand + 8;                        // [2][4]: the exponentials of a tile
  uint64_t* xbar = turn + 8;                        // [4]
  uint64_t* mma_done = xbar + 4;                    // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // the shuffle tells the compiler that a warp has one role
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x & 1;                  // clusters are pairs of neighbours
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); mbar_init(&k_peer[i], 1); }
    for (int i = 0; i < NV; ++i) { mbar_init(&v_full[i], 1); mbar_init(&v_empty[i], 1); mbar_init(&v_peer[i], 1); }
    mbar_init(q_full, LWARPS);
    mbar_init(q_peer, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 8); mbar_init(&pv_done[i], 1); }
    mbar_init(s_empty, 8);
    mbar_init(o_empty, 16);
    for (int i = 0; i < 8; ++i) { mbar_init(&hand[i], 1); mbar_init(&turn[i], 1); }
    for (int i = 0; i < 4; ++i) mbar_init(&xbar[i], 2);
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (EVEN) pdl_launch();                           // the join follows
  tc_fence_before();
  // (without EVEN the walk is of launch constants, not through a structure that
  // the roles' loops would have to read)
  Walk walk{};
  if constexpr (EVEN) walk = uniform(make_walk<M>(x, blockIdx.x >> 1, gridDim.x >> 1, smem));   // in Q's place
  const ItemNo<EVEN> w_first = EVEN ? walk.w : (blockIdx.x >> 1), w_step = EVEN ? walk.step : (gridDim.x >> 1);
  const ItemNo<EVEN> w_last = EVEN ? walk.last : x.n_slots * x.a.hk - 1;
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t per = (uint32_t)a.hq / (uint32_t)a.hk;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, abort_flag, a.err));
  };
  auto wait_pair = [&](uint64_t* bar, uint32_t parity) -> bool {   // arrivals of the other CTA too
    return __all_sync(0xffffffffu, bar_wait<true>(bar, parity, abort_flag, a.err));
  };

  if (warp >= W_LOAD) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
  if (warp >= W_LOAD && warp < W_MMA) {
    // ---------------------------------------------------------------------- Q
    const int lt = tid - 32 * W_LOAD, c = lt & 7, rt = lt >> 3;
    uint32_t items_done = 0;
    for (ItemNo<EVEN> w = w_first; w <= w_last; w += w_step) {
      const Item<M> it = item_of<M, EVEN>(x, walk, w);
      if (it.n_tiles <= 0) continue;
      // once the previous item's last S has read its own
      if (items_done > 0 && !wait(q_empty, (items_done - 1) & 1)) break;
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        const int r = 128 * rank + RT * j + rt;
        const bool valid = r < it.rows;
        const uint32_t f = it.row0 + (valid ? r : 0);
        const uint16_t* src = a.q + it.q_row(a, per, f) * D + 8 * c;
#pragma unroll
        for (int ch = 0; ch < D / 64; ++ch)
          cp_async16_zfill(smem_u32(smem + ch * 16384) + swz128(RT * j + rt, c), src + 64 * ch, valid);
      }
      cp_async_hold(q_full);
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      ++items_done;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == W_TMA) {
    // ---------------------------------------------------------------- K and V
    int ks = 0, vs = 0;
    uint32_t kph = 1, vph = 1, count = 0, k_used = 0, v_used = 0;   // used: stages that copies went to
    bool ok = true;
    const int box = x.box, nb = KT / box, nbk = nb / 2;            // boxes of a tile; of a K half
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
      int id, row, id_v = -1, row_v = 0, id_n, row_n;
      find(it.tile0, id_n, row_n);
      for (int i = 0; ok && i <= it.n_tiles; ++i) {
        id = id_n;
        row = row_n;
        if (i < it.n_tiles) {
          const uint32_t good = __ballot_sync(0xffffffffu, id >= 0);
          reinterpret_cast<volatile uint8_t*>(smem + OFF_OK)[(count % NOK) * 32 + lane] = good >> (4 * lane / box) & 1 ? 15 : 0;
          __syncwarp();                              // every lane's bits before the arrival that lane 0 makes
          ++count;
          if (i + 1 < it.n_tiles) find(it.tile0 + i + 1, id_n, row_n);
          // K: this CTA's 64 keys; lane: box of the half, chunk of 64 dims
          if (!wait(&k_empty[ks], kph)) { ok = false; break; }
          const int kb = rank * nbk + (lane >> 2), ch = lane & 3;
          const int kid = __shfl_sync(0xffffffffu, id, kb & 31), krow = __shfl_sync(0xffffffffu, row, kb & 31);
          const bool mine = lane < 4 * nbk && kid >= 0;
          const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * box * 128;
          if (lane == 0) {
            if (bytes) mbar_arrive_expect_tx(&k_full[ks], bytes);
            else mbar_arrive(&k_full[ks]);
          }
          __syncwarp();
          if (mine)
            tma_load_box(smem_u32(smem + OFF_K + ks * STAGE) + ch * 8192 + (lane >> 2) * box * 128, &x.tk, 64 * ch, krow, it.g,
                         kid, &k_full[ks]);
          if (bytes) k_used |= 1u << ks;
          if (++ks == NK) { ks = 0; kph ^= 1; }
        }
        if (i > 0) {
          // V of the tile before: all 128 keys, this CTA's 128 dims
          if (!wait(&v_empty[vs], vph)) { ok = false; break; }
          const int vb = lane >> 1, c = lane & 1;
          const int vid = __shfl_sync(0xffffffffu, id_v, vb & 31), vrow = __shfl_sync(0xffffffffu, row_v, vb & 31);
          const bool mine = lane < 2 * nb && vid >= 0;
          const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * box * 128;
          if (lane == 0) {
            if (bytes) mbar_arrive_expect_tx(&v_full[vs], bytes);
            else mbar_arrive(&v_full[vs]);
          }
          __syncwarp();
          if (mine)
            tma_load_box(smem_u32(smem + OFF_V + vs * STAGE) + c * 16384 + vb * box * 128, &x.tv, 128 * rank + 64 * c, vrow,
                         it.g, vid, &v_full[vs]);
          if (bytes) v_used |= 1u << vs;
          if (++vs == NV) { vs = 0; vph ^= 1; }
        }
        id_v = id;
        row_v = row;
      }
    }
    // After an abort no TMA copy may still be writing when the CTA exits: wait for
    // the last phase of every stage that one went to.
    if (lane == 0) {
      for (int s = 0; s < NK; ++s)
        if (k_used >> s & 1) mbar_wait_drain(&k_full[s], (s < ks ? kph : kph ^ 1) ^ 1, a.err);
      for (int s = 0; s < NV; ++s)
        if (v_used >> s & 1) mbar_wait_drain(&v_full[s], (s < vs ? vph : vph ^ 1) ^ 1, a.err);
    }
  } else if (warp == W_MMA) {
    // ---------------------------------------------------------------------- S
    int ks = 0;
    uint32_t kph = 0, items_done = 0, count = 0;
    bool ok = true;
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
    for (ItemNo<EVEN> w = w_first; ok && w <= w_last; w += w_step) {
      const Item<M> it = item_of<M, EVEN>(x, walk, w);
      const int n_tiles = __shfl_sync(0xffffffffu, it.n_tiles, 0);
      if (n_tiles <= 0) continue;
      if (!wait(q_full, items_done & 1)) { ok = false; break; }
      fence_async_proxy();                          // written by cp.async, read by the MMA
      if (rank == 1) {
        __syncwarp();
        if (lane == 0) arrive_leader<true>(q_peer);
      } else if (!wait_pair(q_peer, items_done & 1)) {
        ok = false;
        break;
      }
      for (int i = 0; i < n_tiles; ++i, ++count) {
        if (!wait(&k_full[ks], kph)) { ok = false; break; }
        if (rank == 1) {
          fence_async_proxy();
          if (lane == 0) arrive_leader<true>(&k_peer[ks]);
        } else {
          if (!wait_pair(&k_peer[ks], kph)) { ok = false; break; }
          // once the softmax has the scores before in its registers
          if (count > 0 && !wait_pair(s_empty, (count - 1) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t kb = base + OFF_K + ks * STAGE;
#pragma unroll
          for (int e = 0; e < D / 16; ++e)
            umma_ss<2>(tm + TM::s(0), desc_at(DESC_K, base + (e >> 2) * 16384 + 32 * (e & 3)),
                       desc_at(DESC_K, kb + (e >> 2) * 8192 + 32 * (e & 3)), IDESC, e > 0 ? 1u : 0u);
          umma_commit<2>(&k_empty[ks]);
#ifdef QSA_DEBUG_HOOKS
          // test hook: no pair signals its first S, so the softmax times out
          if (!(a.inject == QSA_INJECT_PAGED_STALL && count == 0))
#endif
          umma_commit<2>(&s_full[count & 1]);
          if (i == n_tiles - 1) umma_commit<2>(q_empty);
        }
        if (++ks == NK) { ks = 0; kph ^= 1; }
      }
      ++items_done;
    }
    // every MMA of this warp has retired before TMEM is released (also after an
    // abort: a wait that ignores the flag)
    if (rank == 0) umma_commit<2>(&mma_done[0]);
    mbar_wait_drain(&mma_done[0], 0, a.err);       // in both CTAs: nothing of the first arrives in the second after this
  } else if (warp == W_PV) {
    // -------------------------------------------------------------------- P V
    int vs = 0;
    uint32_t vph = 0, items_done = 0, count = 0;
    bool ok = true;
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
    for (ItemNo<EVEN> w = w_first; ok && w <= w_last; w += w_step) {
      const Item<M> it = item_of<M, EVEN>(x, walk, w);
      const int n_tiles = __shfl_sync(0xffffffffu, it.n_tiles, 0);
      if (n_tiles <= 0) continue;
      for (int i = 0; i < n_tiles; ++i, ++count) {
        if (!wait(&v_full[vs], vph)) { ok = false; break; }
        // rows that no query sees: lane has rows 4 lane .. + 3 of the tile
        {
          uint32_t there = reinterpret_cast<volatile uint8_t*>(smem + OFF_OK)[(count % NOK) * 32 + lane];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int v = (it.tile0 + i) * KT + 4 * lane + k, key = v < it.ns ? v : it.lo + (v - it.ns);
            if (!(v < it.n_vis && (key >= it.first || key < a.sinks))) there &= ~(1u << k);
          }
          if (__any_sync(0xffffffffu, there != 15u)) {
            for (int k = 0; k < 4; ++k)
              if (!(there >> k & 1))
                for (int c = 0; c < 16; ++c)
                  *reinterpret_cast<uint4*>(smem + OFF_V + vs * STAGE + (c >> 3) * 16384 + swz128(4 * lane + k, c & 7)) =
                      make_uint4(0, 0, 0, 0);
            fence_async_proxy();
            __syncwarp();
          }
        }
        if (rank == 1) {
          if (lane == 0) arrive_leader<true>(&v_peer[vs]);
        } else {
          if (!wait_pair(&v_peer[vs], vph) || !wait_pair(&p_full[count & 1], (count >> 1) & 1)) { ok = false; break; }
          if (i == 0 && items_done > 0 && !wait_pair(o_empty, (items_done - 1) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t vb = base + OFF_V + vs * STAGE, p = tm + TM::p(count & 1);
#pragma unroll
          for (int e = 0; e < KT / 16; ++e)
            umma_ts<2>(tm + TM::O, p + 8 * e, desc_at(desc_mn(16384), vb + 2048 * e), IDESC_PV, i > 0 || e > 0 ? 1u : 0u);
          umma_commit<2>(&v_empty[vs]);
          umma_commit<2>(&pv_done[count & 1]);
        }
        if (++vs == NV) { vs = 0; vph ^= 1; }
      }
      ++items_done;
    }
    if (rank == 0) umma_commit<2>(&mma_done[1]);
    mbar_wait_drain(&mma_done[1], 0, a.err);       // in both CTAs: nothing of the first arrives in the second after this
  } else if (warp < W_LOAD) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFT));
    softmax_role<E, D, M, true, EVEN>(x, smem, OFF_OK, OFF_XCH, {s_full, s_empty, p_full, pv_done, hand, turn, xbar, o_empty}, tmem, warp,
                                lane, 128 * rank, walk, w_first, w_last, w_step, blockIdx.x >> 1, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == W_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

template <class E, bool EVEN>
cudaError_t launch_pair(const Args& x, int grid, cudaStream_t s) {
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_done[dev]) {
    e = prepare_launch(paged_prefill_pair_kernel<E, EVEN>, SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev] = true;
  }
  Args y = x;
  y.a.inject = take_debug_injection(QSA_INJECT_PAGED_STALL);
  paged_prefill_pair_kernel<E, EVEN><<<grid, THREADS, SMEM, s>>>(y);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_prefill_pair(const PagedAttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int dtype,
                                      int64_t n_slots, int pairs, bool even, cudaStream_t s) {
  Args x;
  x.tk = tk;
  x.tv = tv;
  x.a = a;
  x.n_slots = n_slots;
  x.box = paged_prefill_box(a.kv.page_size);
  if (dtype == QSA_DTYPE_BF16)
    return even ? launch_pair<__nv_bfloat16, true>(x, 2 * pairs, s) : launch_pair<__nv_bfloat16, false>(x, 2 * pairs, s);
  return even ? launch_pair<__half, true>(x, 2 * pairs, s) : launch_pair<__half, false>(x, 2 * pairs, s);
}

}  // namespace qsa
