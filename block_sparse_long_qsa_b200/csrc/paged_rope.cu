// Norm and rotation of query and key heads, and the append of new tokens to a
// paged cache (qsa_norm_rope, qsa_paged_append).
//
//   y = x / sqrt(mean(x^2) + eps) * w              (per head, fp32)
//   (y_i, y_{i+h}) -> (y_i c - y_{i+h} s, y_{i+h} c + y_i s),  i < h = rope_dim/2
//
// with (c, s) = factor * (cos, sin)(position * f_i), one rounding at the end.
// Bound by HBM: each element is read and written once.
#include "paged.cuh"

namespace qsa {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int UNROLL = 4;     // rows in flight per lane group

// One CTA per token.  A head row is held by D / 8 lanes, 8 dims (16 bytes)
// each; the partner of a rotary pair sits rope_dim / 16 lanes away.  The first
// rows' loads are issued before the angles are formed, so that the two overlap.
template <class E, int D, bool APPEND>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int G = D / 8;                    // lanes of a row
  constexpr int RPW = 32 / G;                 // rows of a warp
  constexpr int STEP = WARPS * RPW;
  using X = Elem<E>;
  __shared__ float2 cs[128];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int l = lane % G, sub = lane / G;
  const int64_t t = blockIdx.x;
  const int n_q = a.q ? a.hq : 0, n_k = a.k ? a.hk : 0;
  const int n_rows = n_q + n_k + (APPEND ? a.hk : 0);   // queries, keys, values

  // ---- where the token goes (append)
  int64_t pos = a.pos0 + t, page_off = -1;
  if (APPEND) {
    int b = (int)t;
    int64_t i = 0;
    if (a.cu_new) {
      b = find_seq(a.cu_new, a.B, t);
      if (b < 0) return;                      // no sequence's row: left as it was
      i = t - a.cu_new[b];
    }
    const int L = a.cache_len[b];
    if (L < 0) return;                        // padding
    pos = (int64_t)L + i;
    if (pos < a.kv.capacity)
      page_off = page_row(a.kv, a.kv.table + (int64_t)b * a.kv.table_ld, (int)pos, tid == 0 ? a.err : nullptr);
    else if (tid == 0)
      report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
  }

  auto src_of = [&](int r) -> const uint16_t* {
    if (r < n_q) return a.q + t * a.q_ld + (int64_t)r * D;
    if (r < n_q + n_k) return a.k + t * a.k_ld + (int64_t)(r - n_q) * D;
    return a.v + t * a.v_ld + (int64_t)(r - n_q - n_k) * D;
  };
  auto dst_of = [&](int r) -> uint16_t* {
    if (r < n_q) return a.q_out + (t * a.hq + r) * D;
    if (!APPEND) return a.k_out + (t * a.hk + (r - n_q)) * D;
    if (page_off < 0) return nullptr;
    const int g = r < n_q + n_k ? r - n_q : r - n_q - n_k;
    return (r < n_q + n_k ? a.kv.k : a.kv.v) + page_off + (int64_t)g * a.kv.head_stride;
  };

  uint4 x[UNROLL] = {};
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int r = base + u * STEP;
      if (r < n_rows) x[u] = *reinterpret_cast<const uint4*>(src_of(r) + 8 * l);
    }
  };
  const int r0 = warp * RPW + sub;
  load(r0);

  const int half = a.rope.half;
  for (int i = tid; i < half; i += THREADS) {
    const int64_t p = a.positions ? (int64_t)a.positions[(int64_t)a.rope.axis[i] * a.T + t] : pos;
    // the angle in half turns, in fp64 (far positions keep their phase), less
    // its whole turns; what is left, at most one, has fp32's precision
    const double turns = (double)p * a.rope.f[i];
    const float rest = (float)(turns - 2.0 * rint(0.5 * turns));
    float s, c;
    sincospif(rest, &s, &c);
    cs[i] = make_float2(a.rope.factor * c, a.rope.factor * s);
  }
  __syncthreads();

  // this lane's pairs and weights
  const int hl = half >> 3;                   // lanes of one half of the rotated dims
  const bool rot = l < 2 * hl;
  const int partner = l < hl ? l + hl : (rot ? l - hl : l);
  const float sign = l < hl ? -1.f : 1.f;
  float c8[8], s8[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 v = rot ? cs[8 * (l < hl ? l : l - hl) + e] : make_float2(1.f, 0.f);
    c8[e] = v.x;
    s8[e] = sign * v.y;
  }
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (a.q_weight) wq = __ldg(reinterpret_cast<const uint4*>(a.q_weight) + l);
  if (a.k_weight) wk = __ldg(reinterpret_cast<const uint4*>(a.k_weight) + l);

  // every lane of a warp takes every step (the shuffles are warp-wide); a row
  // past the last is computed on old registers and not stored
  for (int w0 = warp * RPW; w0 < n_rows; w0 += STEP * UNROLL) {
    if (w0 != warp * RPW) load(w0 + sub);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (w0 + u * STEP >= n_rows) break;
      const int r = w0 + sub + u * STEP;
      const bool is_q = r < n_q, is_v = APPEND && r >= n_q + n_k;
      const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float f[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = X::lo(in[e]);
        f[2 * e + 1] = X::hi(in[e]);
      }
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr) {
        const float inv = rsqrtf(ss * (1.f / D) + a.rope.eps);
        const uint32_t w[4] = {is_q ? wq.x : wk.x, is_q ? wq.y : wk.y, is_q ? wq.z : wk.z, is_q ? wq.w : wk.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[2 * e] *= inv * (X::lo(w[e]) + a.rope.w_plus);
          f[2 * e + 1] *= inv * (X::hi(w[e]) + a.rope.w_plus);
        }
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(0xffffffffu, f[e], partner, G);
        y[e] = rot ? fmaf(o, s8[e], f[e] * c8[e]) : f[e];
      }
      if (r >= n_rows) continue;
      uint16_t* dst = dst_of(r);
      if (!dst) continue;
      uint4 res = x[u];
      if (!is_v)
        res = make_uint4(X::pack(y[0], y[1]), X::pack(y[2], y[3]), X::pack(y[4], y[5]), X::pack(y[6], y[7]));
      *reinterpret_cast<uint4*>(dst + 8 * l) = res;
    }
  }
}

template <class E, bool APPEND>
cudaError_t launch_d(const NormRopeArgs& a, int head_dim, cudaStream_t s) {
  switch (head_dim) {
    case 64: norm_rope_kernel<E, 64, APPEND><<<(unsigned)a.T, THREADS, 0, s>>>(a); break;
    case 128: norm_rope_kernel<E, 128, APPEND><<<(unsigned)a.T, THREADS, 0, s>>>(a); break;
    case 256: norm_rope_kernel<E, 256, APPEND><<<(unsigned)a.T, THREADS, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, int dtype, bool append, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  if (dtype == QSA_DTYPE_BF16)
    return append ? launch_d<__nv_bfloat16, true>(a, head_dim, s) : launch_d<__nv_bfloat16, false>(a, head_dim, s);
  return append ? launch_d<__half, true>(a, head_dim, s) : launch_d<__half, false>(a, head_dim, s);
}

}  // namespace qsa
