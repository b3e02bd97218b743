// Attention of one new token per sequence over its pages (qsa_paged_decode).
//
//   out[b][h] = sum_j softmax_j(q[b][h] . k[j] scale) v[j]
//
// over the keys that window and sinks leave, by one pass with a running maximum
// and sum.  An item is (sequence, KV head, 16 of its query heads): 16 query rows
// against the sequence's visible keys.  Bound by HBM: K and V are read once,
// 4 D bytes a key against 4 D flops a query head.
//
// Split: all items' visible keys are laid end to end in units of a tile a warp and
// cut evenly over the CTAs (one to an SM), so a batch of any mix of lengths
// keeps every SM busy to the last unit.  A CTA's piece of an item that it
// shares with others goes to the scratch as normalised fp32 rows with their
// log-sum-exp; the join kernel adds the pieces in the order of the keys.
//
// Tiles: each warp streams its own KT keys of a unit (head dim 256: 4 warps of 16
// keys; else 8 warps of 2048 / D) through its own ring of three slots with
// cp.async, so no barrier stands between loads and products, and up to 192 KB an
// SM are in flight.  The
// rows are few (M = 16 of mma.sync; a tcgen05 tile of 128 rows would be mostly
// padding) and the products take a third of the time of the loads.
//
// Measured (24 query and 2 KV heads of 256): 64 sequences of 16K to 256K keys
// 1.66 ms in a replayed graph, 1.87 as single calls on fresh inputs, 7.0 and 6.3 TB/s;
// 128 with a window of 4096 keys 148 us, 5.6 TB/s; one of 509 keys 9.5 us, all of it
// latency (two launches, a unit's loads, the join).  32 + 8 heads of 128, 37 sequences
// of up to 32K keys: 162 us, 5.4 TB/s.  Heads of 64: 16 + 16, 40 sequences of up to 40K
// keys 367 to 376 us, 5.0 to 5.1 TB/s; 40 + 5, 64 sequences 158 us, 5.5 TB/s.  40 query
// heads of 64 on one KV head, of which an item takes 16, so the keys are read three
// times: 174 us where one reading takes 57.
#include <cfloat>
#include <type_traits>

#include "paged.cuh"

namespace qsa {
namespace {

constexpr int STAGES = 3;
constexpr int MAX_WARPS = 8;
// Warps of a CTA and bytes of a slot (K and V of KT keys): eight warps hide the
// products' latencies better than four; head dim 256 has four, since a tile of 16
// keys fills 16 KB there.
__host__ __device__ constexpr int warps_of(int D) { return D == 256 ? 4 : 8; }
constexpr int RING = 196608;                      // all slots
constexpr int ROWS = 16;
constexpr int MAX_CTAS = 160;                     // bound of the scratch (148 SMs on B200)
constexpr int MAX_B = 4096;
// The weights are held times 2^shift.  In fp16, whose normal numbers end at 2^-14,
// a first key that outweighs the others would else leave them few bits, and none
// below 2^-25 of its weight; the largest, 2^15, still fits.
template <class E>
constexpr float P_SHIFT = std::is_same<E, __half>::value ? 15.f : 0.f;
constexpr uint32_t OFF_Q = RING;                  // 16 rows of queries
constexpr uint32_t OFF_P = OFF_Q + ROWS * 512;    // running units of the sequences, MAX_B + 1
constexpr uint32_t OFF_V = OFF_P + 4 * (MAX_B + 4);
constexpr uint32_t OFF_ML = OFF_V + MAX_WARPS * STAGES * 8;   // valid rows of each slot above
constexpr uint32_t SMEM = OFF_ML + MAX_WARPS * ROWS * 8 + 64;
static_assert(SMEM <= 232448, "decode smem");

// What CTA c leaves for the join: the item that starts in its range and goes on
// in the next CTAs.
struct JoinRec { int32_t b, hm, last_cta; };

struct Scratch {
  JoinRec* rec;             // [MAX_CTAS]
  float* lse2;              // [2 MAX_CTAS][16] base-2 log-sum-exp
  float* o;                 // [2 MAX_CTAS][16][D]
};
constexpr size_t REC_BYTES = 2048, LSE_BYTES = 2 * MAX_CTAS * ROWS * 4;
static_assert(MAX_CTAS * sizeof(JoinRec) <= REC_BYTES, "join records");
__host__ __device__ inline Scratch scratch_of(void* p) {
  uint8_t* u = static_cast<uint8_t*>(p);
  return {reinterpret_cast<JoinRec*>(u), reinterpret_cast<float*>(u + REC_BYTES),
          reinterpret_cast<float*>(u + REC_BYTES + LSE_BYTES)};
}

// The keys that the token at position L sees, numbered 0 .. n - 1 without the
// gap between sinks and window.
struct Visible {
  int n, ns, lo;
  __device__ __forceinline__ Visible(const PagedAttnArgs& a, int L, uint32_t* err) {
    if (L < 0) { n = ns = lo = 0; return; }
    const bool past = L >= a.kv.capacity;         // past the table: what it holds
    const int end = past ? a.kv.capacity : L + 1;
    if (past) report_error(err, QSA_ERR_DEVICE_BOUNDS);
    lo = a.window > 0 && L >= a.window ? L - a.window + 1 : 0;
    if (lo > end) lo = end;
    ns = a.sinks < lo ? a.sinks : lo;
    n = ns + end - lo;
  }
  __device__ __forceinline__ int key(int v) const { return v < ns ? v : lo + (v - ns); }
};

template <class E, int D>
__global__ void __launch_bounds__(32 * warps_of(D), 1) paged_decode_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int WARPS = warps_of(D), THREADS = 32 * WARPS;
  constexpr int SLOT = RING / (WARPS * STAGES), KT = SLOT / (4 * D);   // a warp's tile
  constexpr int UNIT = WARPS * KT;
  constexpr int G = D / 8;                        // 16-byte chunks of a row
  // copies: LPR lanes a row at a time, so a lane has J rows of a tile, each in CC steps
  constexpr int LPR = D == 256 ? 8 : 4, RPI = 32 / LPR, J = KT / RPI, CC = G / LPR;
  constexpr int NK = KT / 8, NO = D / 8;
  using X = Elem<E>;
  extern __shared__ __align__(1024) uint8_t smem[];
  int32_t* P = reinterpret_cast<int32_t*>(smem + OFF_P);
  uint64_t* vmask = reinterpret_cast<uint64_t*>(smem + OFF_V);
  float2* ml = reinterpret_cast<float2*>(smem + OFF_ML);      // [WARPS][16] running max, sum
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch();

  // ---- units of each sequence (one KV head), summed up: P[b] .. P[b + 1]
  {
    int32_t* wsum = reinterpret_cast<int32_t*>(smem + SMEM - 64);
    int32_t run = 0;
    for (int b0 = 0; b0 < a.B; b0 += THREADS) {
      const int b = b0 + tid;
      int u = 0;
      if (b < a.B) {
        const int L = a.cache_len[b];
        // at least one unit: a row whose keys all lie past the table comes out zero
        if (L >= 0) u = max((Visible(a, L, a.err).n + UNIT - 1) / UNIT, 1);
      }
      int s = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
      if (lane == 31) wsum[warp] = s;
      __syncthreads();
      int before = run, total = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
      }
      if (b < a.B) P[b + 1] = before + s;
      run += total;
      __syncthreads();
    }
    if (tid == 0) P[0] = 0;
    __syncthreads();
  }
  const int per = a.hq / a.hk, MT = (per + ROWS - 1) / ROWS, HM = a.hk * MT;
  const int64_t total = (int64_t)P[a.B] * HM;
  // CTAs that take part: no more than there are units, so none is without one
  const int n_cta = (int)min((int64_t)gridDim.x, total);
  const bool part = (int)blockIdx.x < n_cta;
  const EvenCut cut(total, max(n_cta, 1));
  const int64_t ua = part ? cut.begin(blockIdx.x) : 0, ub = part ? cut.begin(blockIdx.x + 1) : 0;
  Scratch sc = scratch_of(a.scratch);
  if (tid == 0) sc.rec[blockIdx.x] = {0, 0, -1};

  // ---- a position in the laid out units
  struct At {
    int b;                  // sequence
    int hm, u, nu;          // item of the sequence, unit, units of an item
  };
  auto locate = [&](int64_t x) -> At {            // x < total
    int lo = 0, hi = a.B;                         // the b with P[b] HM <= x < P[b + 1] HM
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)P[mid] * HM <= x) lo = mid; else hi = mid;
    }
    const int nu = P[lo + 1] - P[lo];
    const int64_t r = x - (int64_t)P[lo] * HM;
    const int hm = (int)div64(r, nu);
    return {lo, hm, (int)(r - (int64_t)hm * nu), nu};
  };
  auto next_item = [&](At& p) {                   // first unit of the item after p's
    p.u = 0;
    if (++p.hm == HM) {
      p.hm = 0;
      do { ++p.b; } while (p.b < a.B && P[p.b + 1] == P[p.b]);
      if (p.b < a.B) p.nu = P[p.b + 1] - P[p.b];
    }
  };

  // ---- loads: one tile of this warp per unit, in the order of the units.  Few
  // lanes share a row, so a lane has few rows of a tile and finds their places by
  // itself; their page ids are loaded a tile ahead.
  const int cl = lane % LPR, rr = lane / LPR;
  At ia{0, 0, 0, 1};
  int64_t ix = ua;
  int islot = 0;
  Visible iv(a, -1, nullptr);
  const int32_t* itab = a.kv.table;
  int ids[J];
  auto load_ids = [&](bool new_item) {
    if (new_item) {
      iv = Visible(a, __ldg(a.cache_len + ia.b), nullptr);
      itab = a.kv.table + (int64_t)ia.b * a.kv.table_ld;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int v = min(ia.u * UNIT + warp * KT + RPI * j + rr, iv.n - 1);   // past the last: its page
      ids[j] = __ldg(itab + page_of(a.kv, (uint32_t)min(iv.key(max(v, 0)), a.kv.capacity - 1)));
    }
  };
  if (ua < ub) {
    ia = locate(ua);
    load_ids(true);
  }
  At ca = ia;                                      // where the products are
  const uint32_t ring = smem_u32(smem) + warp * STAGES * SLOT;
  // strides in 16-byte units fit 32 bits (checked on the host)
  const uint32_t page16 = (uint32_t)(a.kv.page_stride >> 3), token16 = (uint32_t)(a.kv.token_stride >> 3);
  // row RPI j + rr, chunk LPR cc + cl: row_chunk's exchange is (cl ^ rr) and a 4
  // for every other j (eight lanes a row) or cc (four)
  const uint32_t lane_dst = rr * (D * 2) + ((cl ^ rr) << 4);
  auto issue = [&]() {
    if (ix < ub) {
      const int v0 = ia.u * UNIT + warp * KT + rr;
      const uint32_t kd = ring + islot * SLOT;
      const int64_t head = (int64_t)(ia.hm / MT) * a.kv.head_stride + 8 * cl;
      const uint16_t* kh = a.kv.k + head;
      const uint16_t* vh = a.kv.v + head;
      uint32_t ok = 0;                                              // bit j: row RPI j + rr
      bool bad = false;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int v = v0 + RPI * j, key = iv.key(v);
        const bool there = v < iv.n, good = there && (uint32_t)ids[j] < (uint32_t)a.kv.n_pages;
        bad |= there && !good;
        ok |= (uint32_t)good << j;
        const uint32_t in_page = (uint32_t)key - page_of(a.kv, (uint32_t)key) * (uint32_t)a.kv.page_size;
        const uint64_t off = good ? ((uint64_t)(uint32_t)ids[j] * page16 + (uint64_t)in_page * token16) << 3 : 0;
#pragma unroll
        for (int cc = 0; cc < CC; ++cc) {
          const uint32_t dst = kd + (lane_dst ^ ((LPR == 8 ? j & 1 : cc & 1) << 6)) + RPI * j * (D * 2) +
                               (LPR * cc / 8) * 128;
          cp_async16_zfill(dst, kh + off + 8 * LPR * cc, good);
          cp_async16_zfill(dst + KT * D * 2, vh + off + 8 * LPR * cc, good);
        }
      }
      if (bad) report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
      uint64_t mask = ~0ull;
      if (!__all_sync(0xffffffffu, ok == (uint32_t)((1ull << J) - 1))) {
        mask = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {                               // one bit of each row's lanes, side by side
          uint32_t b = __ballot_sync(0xffffffffu, ok >> j & 1);
          if (LPR == 8) {
            b = (b & 1) | (b >> 7 & 2) | (b >> 14 & 4) | (b >> 21 & 8);
          } else {
            b &= 0x11111111u;
            b = (b | b >> 3) & 0x03030303u;
            b = (b | b >> 6) & 0x000f000fu;
            b = (b | b >> 12) & 0xffu;
          }
          mask |= (uint64_t)b << (RPI * j);
        }
        if (KT < 64) mask |= ~0ull << (KT & 63);
      }
      if (lane == 0) vmask[warp * STAGES + islot] = mask;
      ++ix;
      bool next = ++ia.u == ia.nu;
      if (next) next_item(ia);
      if (ix < ub) load_ids(next);
      if (++islot == STAGES) islot = 0;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES; ++i) issue();

  // ---- products
  const uint32_t q_base = smem_u32(smem) + OFF_Q;
  int slot = 0;
  for (int64_t x = ua; x < ub;) {
    const int n_units = (int)min((int64_t)(ca.nu - ca.u), ub - x);
    const bool whole = n_units == ca.nu;
    const int g = ca.hm / MT, mt = ca.hm % MT;
    const int rows = min(ROWS, per - mt * ROWS);
    const int64_t qrow = (int64_t)ca.b * a.hq + g * per + mt * ROWS;
    // queries of this item (rows past the last are zero)
    for (int e = tid; e < ROWS * G; e += THREADS) {
      const int r = e / G, c = e % G;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows) v = __ldg(reinterpret_cast<const uint4*>(a.q + (qrow + r) * D) + c);
      *reinterpret_cast<uint4*>(smem + OFF_Q + row_chunk<D>(r, c)) = v;
    }
    __syncthreads();
    // up to 128 dims the queries stay in registers
    constexpr bool QREG = D <= 128;
    const uint32_t qr = (lane & 7) + ((lane >> 3) & 1) * 8;
    uint32_t qf[QREG ? D / 16 : 1][4];
    if (QREG)
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) ldsm4(qf[ks], q_base + row_chunk<D>(qr, 2 * ks + (lane >> 4)));

    float o[NO][4];
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // rows lane / 4 and lane / 4 + 8
    int last_slot = 0;
    for (int i = 0; i < n_units; ++i) {
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      const uint64_t ok = vmask[warp * STAGES + slot];
      const uint32_t kd = smem_u32(smem) + (warp * STAGES + slot) * SLOT, vd = kd + KT * D * 2;
      // (bits past the tile are set; no key at all: nothing to add)
      if (KT == 64 ? ok != 0 : (ok & ((1ull << (KT & 63)) - 1)) != 0) {
        // two sums a score where a tile has few: shorter chains of products
        constexpr int CH = NK == 2 ? 2 : 1;
        float sp[CH][NK][4];
#pragma unroll
        for (int n = 0; n < CH * NK; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sp[n / NK][n % NK][e] = 0.f;
        const uint32_t kr = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t (&qa)[4] = qf[QREG ? ks : 0];
          if (!QREG) ldsm4(qa, q_base + row_chunk<D>(qr, 2 * ks + (lane >> 4)));
#pragma unroll
          for (int n = 0; n < NK; n += 2) {
            uint32_t kb[4];
            ldsm4(kb, kd + row_chunk<D>(8 * n + kr, 2 * ks + ((lane >> 3) & 1)));
            X::mma(sp[ks % CH][n], qa, kb[0], kb[1]);
            X::mma(sp[ks % CH][n + 1], qa, kb[2], kb[3]);
          }
        }
        float (&s)[NK][4] = sp[0];
        if (CH == 2)
#pragma unroll
          for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] += sp[CH - 1][n][e];
        if (ok != ~0ull) {
#pragma unroll
          for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((ok >> (8 * n + 2 * (lane & 3) + e)) & 1)) s[n][e] = s[n][e + 2] = -INFINITY;
        }
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          t0 = fmaxf(t0, fmaxf(s[n][0], s[n][1]));
          t1 = fmaxf(t1, fmaxf(s[n][2], s[n][3]));
        }
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
        }
        t0 *= a.scale_log2;
        t1 *= a.scale_log2;
        // the accumulator is rescaled only on tiles that raise some row's maximum
        if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1)) {
          const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
          // a row of nothing but -inf scores keeps the maximum -inf: no factor then
          const float c0 = n0 == -INFINITY ? 1.f : exp2_approx(m0 - n0);
          const float c1 = n1 == -INFINITY ? 1.f : exp2_approx(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= c0;
          l1 *= c1;
#pragma unroll
          for (int n = 0; n < NO; ++n) {
            o[n][0] *= c0;
            o[n][1] *= c0;
            o[n][2] *= c1;
            o[n][3] *= c1;
          }
        }
        const float s0 = (m0 == -INFINITY ? 0.f : m0) - P_SHIFT<E>, s1 = (m1 == -INFINITY ? 0.f : m1) - P_SHIFT<E>;
        // p <= 2^P_SHIFT; the sum takes the fp32 values, the products p rounded to 16 bits
        // (relative error half an ulp of the type, as for the inputs themselves)
        uint32_t pa[KT / 16][4];
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          const float p0 = exp2_approx(fmaf(s[n][0], a.scale_log2, -s0));
          const float p1 = exp2_approx(fmaf(s[n][1], a.scale_log2, -s0));
          const float p2 = exp2_approx(fmaf(s[n][2], a.scale_log2, -s1));
          const float p3 = exp2_approx(fmaf(s[n][3], a.scale_log2, -s1));
          l0 += p0 + p1;
          l1 += p2 + p3;
          pa[n >> 1][(n & 1) * 2] = X::pack(p0, p1);
          pa[n >> 1][(n & 1) * 2 + 1] = X::pack(p2, p3);
        }
        const uint32_t vr = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk) {
#pragma unroll
          for (int n = 0; n < NO; n += 2) {
            uint32_t vb[4];
            ldsm4_t(vb, vd + row_chunk<D>(16 * kk + vr, n + (lane >> 4)));
            X::mma(o[n], pa[kk], vb[0], vb[1]);
            X::mma(o[n + 1], pa[kk], vb[2], vb[3]);
          }
        }
      }
      __syncwarp();                                // the slot is free
      last_slot = slot;
      if (++slot == STAGES) slot = 0;
      if (i + 1 < n_units) issue();                // the last one's slot serves the merge first
    }

    // ---- merge of the warps' rows, each through the slot it used last
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    float* mine = reinterpret_cast<float*>(smem + (warp * STAGES + last_slot) * SLOT);
    const int r0 = lane >> 2, col = 2 * (lane & 3);
    if ((lane & 3) == 0) {
      ml[warp * ROWS + r0] = make_float2(m0, l0);
      ml[warp * ROWS + r0 + 8] = make_float2(m1, l1);
    }
#pragma unroll
    for (int n = 0; n < NO; ++n) {                 // columns exchanged by the row: no bank conflicts
      const int c = (8 * n + col) ^ ((r0 & 7) << 3);
      *reinterpret_cast<float2*>(mine + r0 * D + c) = make_float2(o[n][0], o[n][1]);
      *reinterpret_cast<float2*>(mine + (r0 + 8) * D + c) = make_float2(o[n][2], o[n][3]);
    }
    __syncthreads();
    const int64_t item0 = x - ca.u;                // the item's first unit
    // pieces of an item: 2c + 1 where it starts in CTA c, 2c where it came in from before
    const int piece = 2 * blockIdx.x + (item0 >= ua ? 1 : 0);
    if (tid < rows) {                              // each warp's share of a row, and the row's log-sum-exp
      float mx = -INFINITY, l = 0.f, f[WARPS];
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, ml[w * ROWS + tid].x);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 s = ml[w * ROWS + tid];
        f[w] = s.x == -INFINITY ? (s.y == 0.f ? 0.f : 1.f) : exp2_approx(s.x - mx);
        l = fmaf(f[w], s.y, l);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;  // no key at all: zero
#pragma unroll
      for (int w = 0; w < WARPS; ++w) ml[w * ROWS + tid].x = f[w] * inv;
      const float lse2 = l == 0.f ? -INFINITY : mx + log2f(l) - P_SHIFT<E>;
      if (!whole) sc.lse2[piece * ROWS + tid] = lse2;
      else if (a.lse) a.lse[qrow + tid] = lse2 * 0.69314718055994531f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS * (D / 4) / THREADS; ++i) {
      const int e = i * THREADS + tid, r = e / (D / 4), c = 4 * (e % (D / 4));
      if (r >= rows) break;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = ml[w * ROWS + r].x;
        const float4 v = *reinterpret_cast<const float4*>(smem + (w * STAGES + last_slot) * SLOT +
                                                          (r * D + (c ^ ((r & 7) << 3))) * 4);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (whole)
        *reinterpret_cast<uint2*>(a.out + (qrow + r) * D + c) = make_uint2(X::pack(acc.x, acc.y), X::pack(acc.z, acc.w));
      else
        *reinterpret_cast<float4*>(sc.o + ((int64_t)piece * ROWS + r) * D + c) = acc;
    }
    if (!whole && item0 >= ua && tid == 0)         // and the CTA that has the item's last unit
      sc.rec[blockIdx.x] = {ca.b, ca.hm, (int32_t)cut.owner(item0 + ca.nu - 1)};
    __syncthreads();
    issue();                                       // the merge's slot is free
    x += n_units;
    ca.u += n_units;
    if (ca.u == ca.nu) next_item(ca);
  }
  cp_async_wait<0>();
}

// Joins the pieces of the item that starts in CTA blockIdx.x and goes on after
// it, one query row to a CTA: pieces weighted by 2^(lse - max), in order.
template <class E, int D>
__global__ void __launch_bounds__(256) paged_decode_join_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int C4 = D / 4, GR = 256 / C4;         // threads of a row, pieces at once
  using X = Elem<E>;
  __shared__ float4 acc_s[256];
  __shared__ float2 ml_s[GR];
  pdl_wait();
  const Scratch sc = scratch_of(a.scratch);
  const JoinRec rec = sc.rec[blockIdx.x];
  if (rec.last_cta < 0) return;
  const int per = a.hq / a.hk, MT = (per + ROWS - 1) / ROWS;
  const int g = rec.hm / MT, mt = rec.hm % MT, r = blockIdx.y;
  if (r >= min(ROWS, per - mt * ROWS)) return;
  const int n = rec.last_cta - (int)blockIdx.x + 1;
  const int grp = threadIdx.x / C4, c = 4 * (threadIdx.x % C4);
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = grp; i < n; i += GR) {
    const int64_t piece = 2 * ((int)blockIdx.x + i) + (i == 0 ? 1 : 0);
    const float x = sc.lse2[piece * ROWS + r];
    const float4 v = *reinterpret_cast<const float4*>(sc.o + (piece * ROWS + r) * D + c);
    if (x == -INFINITY) continue;                  // a piece without a key
    const float nm = fmaxf(m, x);
    const float f0 = exp2_approx(m - nm), f1 = exp2_approx(x - nm);
    l = fmaf(l, f0, f1);
    acc.x = fmaf(acc.x, f0, v.x * f1);
    acc.y = fmaf(acc.y, f0, v.y * f1);
    acc.z = fmaf(acc.z, f0, v.z * f1);
    acc.w = fmaf(acc.w, f0, v.w * f1);
    m = nm;
  }
  acc_s[threadIdx.x] = acc;
  if (c == 0) ml_s[grp] = make_float2(m, l);
  __syncthreads();
  if (grp != 0) return;
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < GR; ++i) mx = fmaxf(mx, ml_s[i].x);
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < GR; ++i) {
    const float2 s = ml_s[i];
    const float f = s.y == 0.f ? 0.f : exp2_approx(s.x - mx);
    const float4 v = acc_s[i * C4 + threadIdx.x];
    l = fmaf(f, s.y, l);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t row = (int64_t)rec.b * a.hq + g * per + mt * ROWS + r;
  *reinterpret_cast<uint2*>(a.out + row * D + c) =
      make_uint2(X::pack(acc.x * inv, acc.y * inv), X::pack(acc.z * inv, acc.w * inv));
  if (a.lse && c == 0) a.lse[row] = l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.69314718055994531f;
}

template <class E, int D>
cudaError_t launch_d(const PagedAttnArgs& a, int num_sms, cudaStream_t s, bool join) {
  const int grid = num_sms < MAX_CTAS ? num_sms : MAX_CTAS;
  if (!join) {
    static bool attr_done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !attr_done[dev]) {
      e = cudaFuncSetAttribute(paged_decode_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
      if (e != cudaSuccess) return e;
      if (dev < 64) attr_done[dev] = true;
    }
    paged_decode_kernel<E, D><<<grid, 32 * warps_of(D), SMEM, s>>>(a);
    return cudaGetLastError();
  }
  const int per = a.hq / a.hk;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, per < ROWS ? per : ROWS);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_decode_join_kernel<E, D>, a);
}

}  // namespace

size_t paged_decode_scratch(int head_dim) {
  return REC_BYTES + LSE_BYTES + (size_t)2 * MAX_CTAS * ROWS * head_dim * 4;
}

cudaError_t launch_paged_decode(const PagedAttnArgs& a, int head_dim, int dtype, int num_sms, cudaStream_t s,
                                bool join) {
  if (a.B <= 0) return cudaSuccess;
  if (a.B > MAX_B) return cudaErrorInvalidValue;
  const bool bf = dtype == QSA_DTYPE_BF16;
  switch (head_dim) {
    case 64: return bf ? launch_d<__nv_bfloat16, 64>(a, num_sms, s, join) : launch_d<__half, 64>(a, num_sms, s, join);
    case 128: return bf ? launch_d<__nv_bfloat16, 128>(a, num_sms, s, join) : launch_d<__half, 128>(a, num_sms, s, join);
    case 256: return bf ? launch_d<__nv_bfloat16, 256>(a, num_sms, s, join) : launch_d<__half, 256>(a, num_sms, s, join);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qsa
