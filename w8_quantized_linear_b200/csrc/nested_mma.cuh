// mma.sync fragments of a nested cache's rows: the integer codes are exact in
// fp16, so the tensor cores work on them and the row scales are applied in
// fp32.
#pragma once

#include <math.h>

#include "common.cuh"

namespace bitnest {
namespace nested {

constexpr int kD = 128;  // head dimension (one scale group)

// D = A (16x16 f16, row) * B (16x8 f16, col) + D, fp32
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte codes u of 8 columns from one 32-bit word of each plane: even columns
// (the low nibbles) in `ev`, odd columns in `od`, byte b for plane byte b.
// Draft: u = hi nibble; target: u = (hi << 4) | lo.
template <int MODE>
__device__ __forceinline__ void codes(uint32_t hw, uint32_t lw, uint32_t &ev, uint32_t &od) {
  if (MODE == 0) {
    ev = hw & 0x0F0F0F0Fu;
    od = (hw >> 4) & 0x0F0F0F0Fu;
  } else {
    ev = ((hw << 4) & 0xF0F0F0F0u) | (lw & 0x0F0F0F0Fu);
    od = (hw & 0xF0F0F0F0u) | ((lw >> 4) & 0x0F0F0F0Fu);
  }
}

// fp16 pair (byte b of x, byte b of y) as codes u - offset: 0x6400 | u is the
// half 1024 + u, and 1024 + u - (1024 + offset) is exact.
template <int MODE>
__device__ __forceinline__ uint32_t pair(uint32_t x, uint32_t y, int b) {
  const uint32_t sel = (uint32_t)b | ((uint32_t)(b + 4) << 8);
  const uint32_t t = (prmt(x, y, sel) & 0x00FF00FFu) | 0x64006400u;
  constexpr uint32_t kOff = MODE ? 0xE488E488u : 0xE408E408u;  // -(1024 + offset)
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(kOff));
  return r;
}

// Eight columns (one word of each plane) as fp16 codes in the order 0 2 4 6 1 3 5 7.
template <int MODE>
__device__ __forceinline__ uint4 codes8(uint32_t hw, uint32_t lw) {
  uint32_t ev, od;
  codes<MODE>(hw, lw, ev, od);
  constexpr uint32_t kOff = MODE ? 0xE488E488u : 0xE408E408u;  // -(1024 + offset)
  uint4 r;
  const uint32_t t[4] = {prmt(ev, 0x64646464u, 0x4140), prmt(ev, 0x64646464u, 0x4342),
                         prmt(od, 0x64646464u, 0x4140), prmt(od, 0x64646464u, 0x4342)};
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r.x) : "r"(t[0]), "r"(kOff));
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r.y) : "r"(t[1]), "r"(kOff));
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r.z) : "r"(t[2]), "r"(kOff));
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r.w) : "r"(t[3]), "r"(kOff));
  return r;
}

// pair(x, y, b) and pair(x, y, b + 1)
template <int MODE>
__device__ __forceinline__ void pair2(uint32_t (&r)[2], uint32_t x, uint32_t y, int b) {
  const uint32_t z = prmt(x, y, b ? 0x7362u : 0x5140u);  // x_b, y_b, x_b+1, y_b+1
  constexpr uint32_t kOff = MODE ? 0xE488E488u : 0xE408E408u;  // -(1024 + offset)
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r[0]) : "r"(prmt(z, 0x64646464u, 0x4140)), "r"(kOff));
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r[1]) : "r"(prmt(z, 0x64646464u, 0x4342)), "r"(kOff));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// v as a sum of two fp16 terms, 22 bits together (v below 2^15, and no less than
// 2^-25 of it is kept); `lo` is the second.
__device__ __forceinline__ uint32_t split_half2(float v0, float v1, uint32_t &lo) {
  const uint32_t hi = pack_half2(v0, v1);
  const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  lo = pack_half2(v0 - h.x, v1 - h.y);
  return hi;
}

__device__ __forceinline__ float half_bits(uint16_t b) { return __half2float(__ushort_as_half(b)); }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Query rows of one KV head j: row r is query r >> lgG of the tile's first
// query bi0 (a query is one token of one sequence) and head (j << lgG) + its low
// lgG bits.
__device__ __forceinline__ int64_t query_row(int bi0, int r, int lgG, int H, int j) {
  return (int64_t)(bi0 + (r >> lgG)) * H + (j << lgG) + (r & ((1 << lgG) - 1));
}

// The A operand of the scores for row gid (p0) and gid + 8 (p1) of a 16-row
// tile (null: zeros): k-step ks, K slots 2 tig, 2 tig + 1 <- columns
// 32 tig + 4 ks + {0, 1}, slots 2 tig + 8, 2 tig + 9 <- + {2, 3}; a lane's
// columns are then one 16-byte piece of each plane row.
__device__ __forceinline__ void load_queries(uint32_t (&qa)[8][4], const uint16_t *p0,
                                             const uint16_t *p1, int tig) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    const uint4 a = p0 ? __ldg(reinterpret_cast<const uint4 *>(p0 + 32 * tig) + i) : z;
    const uint4 b = p1 ? __ldg(reinterpret_cast<const uint4 *>(p1 + 32 * tig) + i) : z;
    qa[2 * i][0] = a.x;
    qa[2 * i][1] = b.x;
    qa[2 * i][2] = a.y;
    qa[2 * i][3] = b.y;
    qa[2 * i + 1][0] = a.z;
    qa[2 * i + 1][1] = b.z;
    qa[2 * i + 1][2] = a.w;
    qa[2 * i + 1][3] = b.w;
  }
}

// ... in shared memory (kFrag bytes) for the codes8 operand: columns 0 2 4 6 1 3
// 5 7 of each 8, the even ones in k-step 2 w, the odd ones in 2 w + 1.
constexpr int kFrag = 8 * 32 * 16;
__device__ __forceinline__ void store_frag(uint4 *frag, const uint32_t (&qa)[8][4], int lane) {
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      const uint32_t sel = odd ? 0x7632u : 0x5410u;
      frag[(2 * w + odd) * 32 + lane] =
          make_uint4(prmt(qa[2 * w][0], qa[2 * w][2], sel), prmt(qa[2 * w][1], qa[2 * w][3], sel),
                     prmt(qa[2 * w + 1][0], qa[2 * w + 1][2], sel),
                     prmt(qa[2 * w + 1][1], qa[2 * w + 1][3], sel));
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}

}  // namespace nested
}  // namespace bitnest
