// warp_mma.cuh -- a warp's own copies and products (decode kernels whose warps stream
// tiles by themselves): cp.async, ldmatrix, m16n8k16 with bf16 operands.
#pragma once

#include <stdint.h>

#include "pkv_common.cuh"

namespace pkv {

// 16-byte asynchronous copy; zeros instead when !take.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool take, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(take ? 16 : 0), "l"(policy)
               : "memory");
}
__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// d (16 x 8, fp32) += a (16 x 16, bf16) * b (16 x 8, bf16)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A weight p >= 0 as the sum of two bf16 for a product with V: cut (not rounded), and what that
// leaves, rounded, off by 2^-16 of the weight.  Two weights at a time, packed.  What the cut
// leaves is taken of p and 2^-23 of it, fma(p, kAboveCut, -cut), and so above zero (from p =
// 2^-110 on; 0 of p = 0): a second part of zero or below would make NaN of an infinite value,
// whose product with the first is right.
constexpr float kAboveCut = 1.f + 0x1p-23f;
__device__ __forceinline__ uint32_t cut_bf16x2(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ uint32_t rest_bf16x2(float lo, float hi, uint32_t cut) {
  return pack_bf16x2(fmaf(lo, kAboveCut, -bf16lo(cut)), fmaf(hi, kAboveCut, -bf16hi(cut)));
}

// Byte offset of 16-byte column c of row r in a tile of rows of D values: the
// columns of eight consecutive rows are spread over the banks.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

// The sequence that tile t belongs to (the last s with prefix[s] <= t).
__device__ __forceinline__ int seq_of(const int *prefix, int S, int t) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace pkv
