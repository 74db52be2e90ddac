// mma_common.cuh -- warp-level bf16 matrix products (m16n8k16, fp32 sums) on
// swizzled shared-memory tiles, for the delta-rule kernels.
//
// Their chunk is 64 tokens and most products are 64 x 64 x 64 or 64 x 64 x
// 128, chained one after the other through registers.  Measured on this GPU,
// the warp-level instruction reaches 1018 multiply-adds per cycle per SM (8
// warps) with a latency of 21 cycles; the M = 128 tensor-memory instruction
// at N = 64 gives about 1620 per cycle but only with M = 128 rows to fill,
// and each result passes through tensor memory before the next product can
// use it.
//
// A tile is rows of U 16-byte units; unit u of row r sits at u ^ swz(r), so
// that the eight rows of a matrix fragment fall into different banks.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "tc_common.cuh"

namespace ssd {
namespace mm {

using tc::smem_u32;

template <int U>
__device__ __forceinline__ uint32_t tile_off(int row, int unit) {
  const int x = U >= 8 ? (row & 7) : U == 4 ? ((row >> 1) & 3) : ((row >> 2) & 1);
  return (uint32_t)(row * U + (unit ^ x)) * 16u;
}
// byte offset of element (row, col) of a bf16 tile
template <int U>
__device__ __forceinline__ uint32_t elem_off(int row, int col) {
  return tile_off<U>(row, col >> 3) + (uint32_t)(col & 7) * 2u;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// A fragment of rows m0.., columns k0.. of a tile stored [m][k]
template <int U>
__device__ __forceinline__ void load_a(uint32_t (&r)[4], uint32_t base, int m0, int k0, int lane) {
  ldsm4(r, base + tile_off<U>(m0 + (lane & 15), (k0 >> 3) + (lane >> 4)));
}
// the same of a tile stored [k][m]
template <int U>
__device__ __forceinline__ void load_at(uint32_t (&r)[4], uint32_t base, int m0, int k0, int lane) {
  ldsm4t(r, base + tile_off<U>(k0 + ((lane >> 4) << 3) + (lane & 7), (m0 >> 3) + ((lane >> 3) & 1)));
}
// B fragments of columns n0..n0+15 (two 8-column tiles: r[0..1], r[2..3]),
// k0..k0+15, of a tile stored [n][k]
template <int U>
__device__ __forceinline__ void load_b(uint32_t (&r)[4], uint32_t base, int n0, int k0, int lane) {
  ldsm4(r, base + tile_off<U>(n0 + ((lane >> 4) << 3) + (lane & 7), (k0 >> 3) + ((lane >> 3) & 1)));
}
// the same of a tile stored [k][n]
template <int U>
__device__ __forceinline__ void load_bt(uint32_t (&r)[4], uint32_t base, int n0, int k0, int lane) {
  ldsm4t(r, base + tile_off<U>(k0 + (((lane >> 3) & 1) << 3) + (lane & 7), (n0 >> 3) + (lane >> 4)));
}

// the four 8 x 8 matrices of a fragment back to shared memory
__device__ __forceinline__ void stsm4(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2),
               "r"(r3)
               : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// 16 bytes global -> shared; zeros when `in` is false (src is then not read)
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int K>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(K) : "memory");
}
// R rows of U units from src (row stride in elements), rows >= nvalid as
// zeros, by the nthr threads of one group (tid within the group)
template <int R, int U>
__device__ __forceinline__ void cp_tile(uint32_t dst, const __nv_bfloat16* src, long long stride, int nvalid, int tid,
                                        int nthr) {
#pragma unroll 4
  for (int i = tid; i < R * U; i += nthr) {
    const int r = i / U, u = i % U;
    const bool in = r < nvalid;
    cp16(dst + tile_off<U>(r, u), src + (in ? r * stride + u * 8 : 0), in);
  }
}

// barrier `id` among n threads of the CTA
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

}  // namespace mm
}  // namespace ssd
