// Attention of a ragged batch of new tokens over their pages (qsa_paged_prefill).
//
// Item = (64 query rows of one sequence, KV head); the rows are the sequence's
// (token, query head of the KV head) pairs laid out flat, so every head count
// fills the tiles.  One pass over the visible keys with a running maximum and sum.
#include <cfloat>

#include "paged.cuh"

namespace qsa {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int ROWS = 16 * WARPS;
constexpr int KT = 32;

template <int D>
constexpr uint32_t smem_bytes() {
  return (ROWS + 4 * KT) * D * 2 + 64;
}

template <class E, int D>
__global__ void __launch_bounds__(THREADS) paged_prefill_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int G = D / 8, NK = KT / 8, NO = D / 8;
  using X = Elem<E>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_base = smem_u32(smem), kv_base = q_base + ROWS * D * 2;
  uint32_t* vmask = reinterpret_cast<uint32_t*>(smem + (ROWS + 4 * KT) * D * 2);   // [2]
  const int per = a.hq / a.hk, g = blockIdx.y;
  // Tile slots: sequence b owns the slots from cu[b] per / 64 + b on (at least as
  // many as it has tiles).  The last slots come first.
  const int64_t slot = (int64_t)gridDim.x - 1 - blockIdx.x;
  int b = 0;
  {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)a.cu_new[mid] * per / ROWS + mid <= slot) lo = mid; else hi = mid;
    }
    b = lo;
  }
  const int64_t t0 = a.cu_new[b], t1 = min((int64_t)a.cu_new[b + 1], a.T);
  const int64_t tile = slot - (t0 * per / ROWS + b);
  const int64_t n_rows = (t1 - t0) * per;
  const int L = a.cache_len[b];
  if (t0 < 0 || tile < 0 || tile * ROWS >= n_rows || L < 0) return;
  const int64_t row0 = tile * ROWS;
  const int rows = (int)min((int64_t)ROWS, n_rows - row0);
  // positions of the first and the last row's tokens
  const int64_t p_first = L + row0 / per, p_last = L + (row0 + rows - 1) / per;
  if (p_last >= a.kv.capacity && tid == 0) report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
  const int end = (int)min(p_last + 1, (int64_t)a.kv.capacity);
  int lo = a.window > 0 && p_first >= a.window ? (int)(p_first - a.window + 1) : 0;
  if (lo > end) lo = end;
  const int ns = min(a.sinks, lo), n_vis = ns + end - lo;
  const int n_tiles = (n_vis + KT - 1) / KT;
  const int32_t* table = a.kv.table + (int64_t)b * a.kv.table_ld;

  // queries
  for (int e = tid; e < ROWS * G; e += THREADS) {
    const int r = e / G, c = e % G;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < rows) {
      const int64_t f = row0 + r;
      v = __ldg(reinterpret_cast<const uint4*>(a.q + ((t0 + f / per) * a.hq + g * per + f % per) * D) + c);
    }
    *reinterpret_cast<uint4*>(smem + row_chunk<D>(r, c)) = v;
  }
  auto issue = [&](int i) {
    if (i < n_tiles) {
      const int v = i * KT + lane;
      const int64_t off = v < n_vis ? page_row(a.kv, table, v < ns ? v : lo + (v - ns), a.err) : -1;
      const uint32_t ok = __ballot_sync(0xffffffffu, off >= 0);
      if (tid == 0) vmask[i & 1] = ok;
      const uint32_t kd = kv_base + (i & 1) * 2 * KT * D * 2, vd = kd + KT * D * 2;
#pragma unroll
      for (int j = 0; j < KT * G / THREADS; ++j) {
        const int e = j * THREADS + tid, row = e / G, c = e % G;
        const int64_t o = __shfl_sync(0xffffffffu, off, row) + g * a.kv.head_stride + 8 * c;
        const bool valid = (ok >> row) & 1;
        cp_async16_zfill(kd + row_chunk<D>(row, c), valid ? a.kv.k + o : a.kv.k, valid);
        cp_async16_zfill(vd + row_chunk<D>(row, c), valid ? a.kv.v + o : a.kv.v, valid);
      }
    }
    cp_async_commit();
  };
  issue(0);
  float o[NO][4];
#pragma unroll
  for (int i = 0; i < NO; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int64_t pos[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) pos[h] = L + (row0 + 16 * warp + (lane >> 2) + 8 * h) / per;
  for (int i = 0; i < n_tiles; ++i) {
    issue(i + 1);
    cp_async_wait<1>();
    __syncthreads();
    const uint32_t ok = vmask[i & 1];
    const uint32_t kd = kv_base + (i & 1) * 2 * KT * D * 2, vd = kd + KT * D * 2;
    float s[NK][4];
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
    const uint32_t qr = 16 * warp + (lane & 7) + ((lane >> 3) & 1) * 8, kr = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t qa[4];
      ldsm4(qa, q_base + row_chunk<D>(qr, 2 * ks + (lane >> 4)));
#pragma unroll
      for (int n = 0; n < NK; n += 2) {
        uint32_t kb[4];
        ldsm4(kb, kd + row_chunk<D>(8 * n + kr, 2 * ks + ((lane >> 3) & 1)));
        X::mma(s[n], qa, kb[0], kb[1]);
        X::mma(s[n + 1], qa, kb[2], kb[3]);
      }
    }
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 8 * n + 2 * (lane & 3) + (e & 1), v = i * KT + c;
        const int key = v < ns ? v : lo + (v - ns);
        const int64_t ps = pos[e >> 1];
        const bool seen = ((ok >> c) & 1) && key <= ps && (a.window == 0 || key > ps - a.window || key < a.sinks);
        if (!seen) s[n][e] = -INFINITY;
      }
    float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e >> 1] = fmaxf(t[e >> 1], s[n][e]);
    float base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      t[h] = fmaxf(t[h], __shfl_xor_sync(0xffffffffu, t[h], 1));
      t[h] = fmaxf(t[h], __shfl_xor_sync(0xffffffffu, t[h], 2)) * a.scale_log2;
      const float nm = fmaxf(m[h], t[h]);
      const float f = nm == -INFINITY ? 1.f : exp2_approx(m[h] - nm);
      m[h] = nm;
      l[h] *= f;
#pragma unroll
      for (int n = 0; n < NO; ++n) {
        o[n][2 * h] *= f;
        o[n][2 * h + 1] *= f;
      }
      base[h] = nm == -INFINITY ? 0.f : nm;
    }
    uint32_t pa[KT / 16][4];
#pragma unroll
    for (int n = 0; n < NK; ++n) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = exp2_approx(fmaf(s[n][e], a.scale_log2, -base[e >> 1]));
        l[e >> 1] += p[e];
      }
      pa[n >> 1][(n & 1) * 2] = X::pack(p[0], p[1]);
      pa[n >> 1][(n & 1) * 2 + 1] = X::pack(p[2], p[3]);
    }
    const uint32_t vr = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
    for (int kk = 0; kk < KT / 16; ++kk)
#pragma unroll
      for (int n = 0; n < NO; n += 2) {
        uint32_t vb[4];
        ldsm4_t(vb, vd + row_chunk<D>(16 * kk + vr, n + (lane >> 4)));
        X::mma(o[n], pa[kk], vb[0], vb[1]);
        X::mma(o[n + 1], pa[kk], vb[2], vb[3]);
      }
    __syncthreads();
  }
  cp_async_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    const int r = 16 * warp + (lane >> 2) + 8 * h;
    if (r >= rows) continue;
    const int64_t f = row0 + r, row = (t0 + f / per) * a.hq + g * per + f % per;
    const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
#pragma unroll
    for (int n = 0; n < NO; ++n)
      *reinterpret_cast<uint32_t*>(a.out + row * D + 8 * n + 2 * (lane & 3)) =
          X::pack(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
    if (a.lse && (lane & 3) == 0)
      a.lse[row] = l[h] == 0.f ? -INFINITY : (m[h] + log2f(l[h])) * 0.69314718055994531f;
  }
}

template <class E, int D>
cudaError_t launch_d(const PagedAttnArgs& a, cudaStream_t s) {
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(paged_prefill_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes<D>());
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev] = true;
  }
  const int64_t slots = (a.T * (a.hq / a.hk) + ROWS - 1) / ROWS + a.B;
  paged_prefill_kernel<E, D><<<dim3((unsigned)slots, a.hk), THREADS, smem_bytes<D>(), s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t paged_prefill_scratch(int) { return 0; }

cudaError_t launch_paged_prefill(const PagedAttnArgs& a, int head_dim, int dtype, int, cudaStream_t s, bool join) {
  if (a.B <= 0 || a.T <= 0 || join) return cudaSuccess;
  const bool bf = dtype == QSA_DTYPE_BF16;
  switch (head_dim) {
    case 64: return bf ? launch_d<__nv_bfloat16, 64>(a, s) : launch_d<__half, 64>(a, s);
    case 128: return bf ? launch_d<__nv_bfloat16, 128>(a, s) : launch_d<__half, 128>(a, s);
    case 256: return bf ? launch_d<__nv_bfloat16, 256>(a, s) : launch_d<__half, 256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qsa
