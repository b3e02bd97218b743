// Shared pieces of the paged-cache kernels: the page table walk, the visible
// keys of a token, 16-bit element conversion, and the warp-level matrix
// instructions of the kernels whose tiles have few rows.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qsa_device.cuh"
#include "paged_index.h"
#include "qsa_kernels.h"

namespace qsa {

// ---------------------------------------------------------------- elements --
// E is __nv_bfloat16 or __half; both travel as 16-bit patterns, two to a word.
template <class E> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
  // round to nearest even; infinities and NaN kept
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <> struct Elem<__half> {
  static __device__ __forceinline__ float lo(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// ------------------------------------------------------------- page tables --
// j / page_size for 0 <= j < 2^31
__device__ __forceinline__ uint32_t page_of(const PagedView& c, uint32_t j) {
  return page_quotient(c.div_mul, c.div_shift, j);
}
// Element offset of token j's row of KV head 0, or -1 where the table entry
// names no page (recorded).  j must lie in [0, c.capacity).
__device__ __forceinline__ int64_t page_row(const PagedView& c, const int32_t* __restrict__ table_row, int j,
                                            uint32_t* err) {
  const uint32_t pg = page_of(c, (uint32_t)j);
  const int32_t id = __ldg(table_row + pg);
  if ((uint32_t)id >= (uint32_t)c.n_pages) {
    report_error(err, QSA_ERR_DEVICE_BOUNDS);
    return -1;
  }
  return (int64_t)id * c.page_stride + (int64_t)(j - (int)(pg * (uint32_t)c.page_size)) * c.token_stride;
}

// The sequence of row t: the last b with cu[b] <= t, or -1 (t before cu[0], or
// behind cu[B]).  One warp, 32 offsets a step; offsets that do not ascend give
// some b in [0, B).
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ cu, int B, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo >= 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < hi && (int64_t)__ldg(cu + i) <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    if (n == 0) return -1;
    lo += (n - 1) * step;
    hi = min(lo + step, hi);
    if (step == 1) break;
  }
  return t < (int64_t)__ldg(cu + B) ? lo : -1;
}

// ------------------------------------------------------ copies and fragments --
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Byte offset of 16-byte chunk c of a row of D elements: the low three bits of
// the chunk are exchanged by the row, so eight rows of one chunk (what ldmatrix
// reads at once) lie in eight different bank groups.
template <int D>
__device__ __forceinline__ uint32_t row_chunk(uint32_t row, uint32_t c) {
  return row * (uint32_t)(D * 2) + ((c ^ (row & 7u)) << 4);
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Programmatic dependent launch: a kernel launched with the attribute may start
// while its predecessor runs; pdl_wait returns once that one has ended and its
// writes are visible.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace qsa
