// Norm and rotation of query and key heads, and the append of new tokens to a
// paged cache (qsa_norm_rope, qsa_paged_append).
//
//   y = x / sqrt(mean(x^2) + eps) * w              (per head, fp32)
//   (y_i, y_{i+h}) -> (y_i c - y_{i+h} s, y_{i+h} c + y_i s),  i < h = rope_dim/2
//
// with (c, s) = factor * (cos, sin)(position * f_i), one rounding at the end.
// Bound by HBM: each element is read and written once (32768 tokens of 24 + 2
// heads of 256: 137 us in a replayed graph, 147 as single calls on fresh inputs, 97
// and 90 % of a plain copy's rate; appended with their values for 13 sequences,
// 24472 tokens in all: 116 and 124 us, 92 and 86 %; 64 tokens: 3 to 5 us, one launch's
// latency).
#include "paged.cuh"

namespace qsa {
namespace {

// Warps of a CTA: one, so that a warp's place is taken as soon as it is done (32K
// tokens of 24 + 2 heads of 256: 136 us, with two warps 145, with four 146).
constexpr int WARPS = 1;
// Rows of a lane group in flight (32K tokens: 2 rows 148 us, 4 rows 136, 6 rows 138).
constexpr int U = 4;
// Below this many tokens a token's rows are spread over several warps (26 rows
// of 256: 2048 tokens 13.7 us against 15.3 with a warp a token, 4096 tokens 24.1
// against 21.2).
constexpr int64_t FEW_TOKENS = 3000;

// A warp takes one token's rows, or with few tokens one step's rows (U per lane
// group) of one of q, k, v.  A head row is held by D / 8 lanes, 8 dims (16 bytes)
// each; the partner of a rotary pair sits rope_dim / 16 lanes away.  With the
// weights folded into the rotation,
//   y = inv (x cw + x' sw),  cw = w c,  sw = -+ w' s  (x', w': the partner's),
// a row costs one shuffle of the raw partner words, the sum of squares, and
// three packed operations a pair of dims.
template <class E, int D, bool APPEND>
__global__ void __launch_bounds__(32 * WARPS) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int G = D / 8;                    // lanes of a row
  constexpr int RPW = 32 / G;                 // rows of a warp
  constexpr int STEP = RPW * U;
  using X = Elem<E>;
  __shared__ float2 cs_all[WARPS][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % G, sub = lane / G;
  const uint32_t unit = blockIdx.x * WARPS + warp;   // T parts < 2^31
  const int64_t t = unit / (uint32_t)a.parts;
  if (t >= a.T) return;
  const int part = (int)(unit - (uint32_t)t * (uint32_t)a.parts);
  float2* cs = cs_all[warp];
  const int n_q = a.q ? a.hq : 0, n_k = a.k ? a.hk : 0, n_v = APPEND ? a.hk : 0;

  // this warp's rows: [q0, q1), [k0, k1), [v0, v1)
  int q0 = 0, q1 = n_q, k0 = 0, k1 = n_k, v0 = 0, v1 = n_v;
  if (a.parts > 1) {
    const int pq = (n_q + STEP - 1) / STEP, pk = (n_k + STEP - 1) / STEP;
    const int iq = part, ik = iq - pq, iv = ik - pk;
    q0 = iq * STEP, q1 = min(q0 + STEP, n_q);             // empty where the part is another's
    k0 = ik < 0 ? n_k : ik * STEP, k1 = min(k0 + STEP, n_k);
    v0 = iv < 0 ? n_v : iv * STEP, v1 = min(v0 + STEP, n_v);
  }

  const uint16_t* q_row = a.q + t * a.q_ld + 8 * l;
  const uint16_t* k_row = a.k + t * a.k_ld + 8 * l;
  const uint16_t* v_row = a.v + t * a.v_ld + 8 * l;
  uint4 x[U] = {};
  auto load = [&](const uint16_t* row, int r0, int r1) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPW + sub;
      if (r < r1) x[u] = *reinterpret_cast<const uint4*>(row + (int64_t)r * D);
    }
  };
  // the first rows are on their way while place and angles are found
  if (q0 < q1) load(q_row, q0, q1);
  else if (k0 < k1) load(k_row, k0, k1);
  else load(v_row, v0, v1);

  // ---- where the token goes (append)
  int64_t pos = a.pos0 + t, page_off = -1;
  if (APPEND) {
    int b = (int)t;
    int64_t i = 0;
    if (a.cu_new) {
      b = find_seq(a.cu_new, a.B, t);
      if (b < 0) return;                      // no sequence's row: left as it was
      i = t - a.cu_new[b];
      if (i < 0) return;                      // offsets that do not ascend
    }
    const int L = a.cache_len[b];
    if (L < 0) return;                        // padding
    pos = (int64_t)L + i;
    if (pos < a.kv.capacity)
      page_off = page_row(a.kv, a.kv.table + (int64_t)b * a.kv.table_ld, (int)pos, lane == 0 ? a.err : nullptr);
    else if (lane == 0)
      report_error(a.err, QSA_ERR_DEVICE_BOUNDS);
  }

  const int half = a.rope.half;
  if (q0 < q1 || k0 < k1) {
    for (int i = lane; i < half; i += 32) {
      const int64_t p = a.positions ? (int64_t)a.positions[(int64_t)a.rope.axis[i] * a.T + t] : pos;
      // the angle in half turns, in fp64 (far positions keep their phase), less
      // its whole turns; what is left, at most one, has fp32's precision
      const double turns = (double)p * a.rope.f[i];
      const float rest = (float)(turns - 2.0 * rint(0.5 * turns));
      float s, c;
      sincospif(rest, &s, &c);
      cs[i] = make_float2(a.rope.factor * c, a.rope.factor * s);
    }
    __syncwarp();
  }

  const int hl = half >> 3;                   // lanes of one half of the rotated dims
  const bool rot = l < 2 * hl;
  const int partner = l < hl ? l + hl : (rot ? l - hl : l);

  // rows [r0, r1) of q or of k to out, out_ld elements apart; x holds the first
  // step's when loaded.  (q and k may be one tensor: nothing goes by their addresses.)
  auto turn = [&](const uint16_t* row, int r0, int r1, const uint16_t* weight, uint16_t* out, int64_t out_ld, bool loaded) {
    if (r0 >= r1) return;
    uint64_t cw[4], sw[4];
    {
      uint4 wo = make_uint4(0, 0, 0, 0), wp = wo;
      if (weight) {
        wo = __ldg(reinterpret_cast<const uint4*>(weight) + l);
        wp = __ldg(reinterpret_cast<const uint4*>(weight) + partner);
      }
      const uint32_t o[4] = {wo.x, wo.y, wo.z, wo.w}, p[4] = {wp.x, wp.y, wp.z, wp.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float w0 = 1.f, w1 = 1.f, p0 = 1.f, p1 = 1.f;
        if (weight) {
          w0 = X::lo(o[e]) + a.rope.w_plus, w1 = X::hi(o[e]) + a.rope.w_plus;
          p0 = X::lo(p[e]) + a.rope.w_plus, p1 = X::hi(p[e]) + a.rope.w_plus;
        }
        float2 a0 = make_float2(1.f, 0.f), a1 = a0;
        if (rot) {
          const float2* c = cs + 8 * (l < hl ? l : l - hl) + 2 * e;
          a0 = c[0], a1 = c[1];
        }
        const float sg = l < hl ? -1.f : 1.f;
        cw[e] = pk2(w0 * a0.x, w1 * a1.x);
        sw[e] = pk2(sg * p0 * a0.y, sg * p1 * a1.y);
      }
    }
    for (int r = r0; r < r1; r += STEP) {
      if (!loaded) load(row, r, r1);
      loaded = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + u * RPW >= r1) break;
        const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        uint64_t f[4], y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e] = pk2(X::lo(in[e]), X::hi(in[e]));
          y[e] = mul2(f[e], cw[e]);
        }
        if (half) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // lanes beyond the rotated dims add nothing, whatever they hold
            const uint32_t o = __shfl_sync(0xffffffffu, in[e], partner, G);
            y[e] = fma2(rot ? pk2(X::lo(o), X::hi(o)) : 0ull, sw[e], y[e]);
          }
        }
        if (weight) {
          uint64_t ss = mul2(f[0], f[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) ss = fma2(f[e], f[e], ss);
          float s0, s1;
          upk2(ss, s0, s1);
          s0 += s1;
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
          const float inv = rsqrtf(s0 * (1.f / D) + a.rope.eps);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], pk2(inv, inv));
        }
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y0, y1;
          upk2(y[e], y0, y1);
          w[e] = X::pack(y0, y1);
        }
        if (out && r + u * RPW + sub < r1)
          *reinterpret_cast<uint4*>(out + (int64_t)(r + u * RPW + sub) * out_ld) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  const bool has_q = q0 < q1, has_k = k0 < k1;
  turn(q_row, q0, q1, a.q_weight, a.q_out + t * a.hq * D + 8 * l, D, true);
  uint16_t* k_out = APPEND ? (page_off >= 0 ? a.kv.k + page_off + 8 * l : nullptr) : a.k_out + t * a.hk * D + 8 * l;
  turn(k_row, k0, k1, a.k_weight, k_out, APPEND ? a.kv.head_stride : D, !has_q);
  if (APPEND && page_off >= 0) {
    bool loaded = !has_q && !has_k;
    for (int r = v0; r < v1; r += STEP) {
      if (!loaded) load(v_row, r, v1);
      loaded = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = r + u * RPW + sub;
        if (h < v1) *reinterpret_cast<uint4*>(a.kv.v + page_off + (int64_t)h * a.kv.head_stride + 8 * l) = x[u];
      }
    }
  }
}

template <class E, int D, bool APPEND>
cudaError_t launch_one(NormRopeArgs a, cudaStream_t s) {
  constexpr int STEP = 32 / (D / 8) * U;
  const int n_q = a.q ? a.hq : 0, n_k = a.k ? a.hk : 0, n_v = APPEND ? a.hk : 0;
  // a warp for each step's rows while the tokens alone do not fill the GPU
  const int parts = (n_q + STEP - 1) / STEP + (n_k + STEP - 1) / STEP + (n_v + STEP - 1) / STEP;
  a.parts = a.T < FEW_TOKENS ? parts : 1;
  const int64_t warps = a.T * a.parts;
  norm_rope_kernel<E, D, APPEND><<<(unsigned)((warps + WARPS - 1) / WARPS), 32 * WARPS, 0, s>>>(a);
  return cudaGetLastError();
}

template <class E, bool APPEND>
cudaError_t launch_d(const NormRopeArgs& a, int head_dim, cudaStream_t s) {
  switch (head_dim) {
    case 64: return launch_one<E, 64, APPEND>(a, s);
    case 128: return launch_one<E, 128, APPEND>(a, s);
    case 256: return launch_one<E, 256, APPEND>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, int dtype, bool append, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  if (dtype == QSA_DTYPE_BF16)
    return append ? launch_d<__nv_bfloat16, true>(a, head_dim, s) : launch_d<__nv_bfloat16, false>(a, head_dim, s);
  return append ? launch_d<__half, true>(a, head_dim, s) : launch_d<__half, false>(a, head_dim, s);
}

}  // namespace qsa
