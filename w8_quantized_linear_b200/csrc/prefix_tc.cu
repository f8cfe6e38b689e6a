// Attention over a shared prefix on tcgen05, for the many rows (queries x
// heads of one KV head) that a batch gives: S = Q K^T and O = P V with 128 x
// 128 tiles, both accumulators in tensor memory, one pass with a running
// maximum.
//
// A CTA takes 256 rows of one KV head (two tiles, A and B) and 128 tokens at a
// time, and an equal run of such units over all KV heads and row groups.  16
// warps:
//   0-7    softmax of tile A (0-3) and B (4-7), one row a thread: the scores
//          from tensor memory, times the tokens' K scales, the row's running
//          maximum, p = 2^(s - shift), times the V scales, rounded to fp16 and
//          written back over the scores as the second product's A operand;
//   8-11   the cache's codes as fp16 operands: plane words -> shared memory
//          (128-byte swizzle), two stages of K and of V; the tokens' scales;
//   12     issues the MMAs.
// The tensor cores work on tile B while A is in its softmax and back.
//
// The codes are exact in fp16, so a score is off by fp32 sums only.  The
// output is rescaled only when a row's maximum has grown by 2^8 or the largest
// V scale has (the softmax warps do it in place): p is kept as 2^(s - shift)
// with shift = m + e - 7, m a maximum that is at most 8 behind, 2^e above every
// V scale so far, so p v_scale < 2^15 in fp16, with 2^29 between it and fp16's
// subnormals; row sums carry the same factor, which cancels.
//
// Columns of a head are kept in the order 0 2 4 6 1 3 5 7 within each 8 (the
// order in which plane words unpack with the fewest instructions): the same
// for Q and K, and undone when the output is written.
#include <math.h>

#include "nested_mma.cuh"
#include "prefix_plan.h"
#include "sm100.cuh"

namespace bitnest {
namespace pattn {

namespace {

using namespace nested;

constexpr int kRowsTile = 128, kRowsCta = 256, kTokens = 128;
constexpr int kThreads = 512;
constexpr int kLaunchRegs = 128;  // 512 threads x 128 = the SM's registers
// after the split: 256 x 184 + 128 x 96 + 128 x 48 = 512 x 128
constexpr int kRegSoftmax = 184, kRegOperand = 96, kRegIssue = 48;
static_assert(2 * kRegSoftmax + kRegOperand + kRegIssue == 4 * kLaunchRegs, "register split");
constexpr int kStages = 2, kSlots = 4;
constexpr int kOperand = kTokens * kD * 2;  // bytes of a K, V or Q tile
constexpr float kScale = 0.088388347648318440550f * 1.4426950408889634f;  // log2(e) / sqrt(128)
constexpr float kSlack = 8.0f;
constexpr int kHead = 7;  // p v_scale < 2^(8 + 7)
constexpr int kMinExp = -40;  // below any fp16 scale / 16

constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 2 * kOperand;
constexpr int kOffV = kOffK + kStages * kOperand;
constexpr int kOffScale = kOffV + kStages * kOperand;        // [slot][k, v][128] floats
constexpr int kOffExp = kOffScale + kSlots * 2 * kTokens * 4;  // [slot][4] ints
constexpr int kOffBar = kOffExp + kSlots * 4 * 4;
constexpr int kBars = 4 * kStages + kSlots + 2 * 4 + 1;
constexpr int kSmem = kOffBar + kBars * 8 + 16 + 1024;

constexpr int kColO = 0, kColS = 256;  // tensor memory columns (tile B: + 128)

// kind::f16 with fp32 accumulation: A fp16 (K-major), B fp16 (K-major, or
// MN-major when bn), 128 x 128
constexpr uint32_t idesc(bool bn) {
  return (1u << 4) | (bn ? 1u << 16 : 0u) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
}

// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}

// MN-major operand, 128-byte swizzle: 64 columns (128 bytes) of one token a
// line, 8 tokens 1024 bytes, the next 64 columns 16 KB on.
__device__ __forceinline__ uint64_t desc_mn_sw128(const void *base) {
  uint64_t d = 0;
  d |= ((uint64_t)smem_u32(base) >> 4) & 0x3FFFull;
  d |= (uint64_t)((kOperand / 2) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void ld32(uint32_t taddr, float *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]),
        "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]),
        "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void st32(uint32_t taddr, const float *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
      "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]),
      "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]), "f"(r[19]), "f"(r[20]), "f"(r[21]),
      "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]),
      "f"(r[29]), "f"(r[30]), "f"(r[31])
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// One thread's share of a tile's plane rows: for q = 0 .. 3, 16 bytes (piece
// tid % 4) of the row of token 32 q + tid / 4.
struct Words {
  uint4 hi[4], lo[4];
};
template <int MODE>
__device__ __forceinline__ void load_words(Words &w, const uint8_t *__restrict__ hi,
                                           const uint8_t *__restrict__ lo, int64_t t0, int64_t P,
                                           int64_t Hkv, int j, int tid) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t t = t0 + 32 * q + (tid >> 2);
    w.hi[q] = w.lo[q] = make_uint4(0, 0, 0, 0);
    if (t < P) {
      const int64_t off = (t * Hkv + j) * (kD / 2) + 16 * (tid & 3);
      w.hi[q] = __ldg(reinterpret_cast<const uint4 *>(hi + off));
      if (MODE) w.lo[q] = __ldg(reinterpret_cast<const uint4 *>(lo + off));
    }
  }
}
// ... as fp16 to the tile at `dst`: token rows of 128 bytes in two halves (64
// columns each, 16 KB apart), 16-byte chunk c of row t at c ^ (t % 8).  Pieces
// 2 and 3 (the second half) take their words in the order 2 3 0 1, so that the
// eight lanes of a store phase fall in different banks.
template <int MODE>
__device__ __forceinline__ void store_words(uint8_t *dst, const Words &w, int tid) {
  const int piece = tid & 3;
  const bool swap = piece >= 2;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int t = 32 * q + (tid >> 2);
    uint8_t *row = dst + (piece >> 1) * (kOperand / 2) + t * 128;
    const uint32_t h[4] = {w.hi[q].x, w.hi[q].y, w.hi[q].z, w.hi[q].w};
    const uint32_t l[4] = {w.lo[q].x, w.lo[q].y, w.lo[q].z, w.lo[q].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t hw = swap ? h[c ^ 2] : h[c], lw = MODE ? (swap ? l[c ^ 2] : l[c]) : 0u;
      const int chunk = ((piece & 1) * 4 + (swap ? c ^ 2 : c)) ^ (t & 7);
      *reinterpret_cast<uint4 *>(row + chunk * 16) = codes8<MODE>(hw, lw);
    }
  }
}

struct Units {  // a CTA's run of units, one row group (item) at a time
  int u, end, tiles;
  __device__ __forceinline__ bool next(int &item, int &t0, int &n) {
    if (u >= end) return false;
    item = u / tiles;
    t0 = u - item * tiles;
    n = min(end - u, tiles - t0);
    u += n;
    return true;
  }
};

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) prefix_tc_kernel(PrefixAttnArgs a, Plan pl,
                                                                float *__restrict__ part_lse,
                                                                float *__restrict__ part_o) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float *scales = reinterpret_cast<float *>(sm + kOffScale);
  int *exps = reinterpret_cast<int *>(sm + kOffExp);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kOffBar);
  uint64_t *k_full = bars, *k_free = k_full + kStages, *v_full = k_free + kStages,
           *v_free = v_full + kStages, *sc_full = v_free + kStages, *q_full = sc_full + kSlots,
           *s_full = q_full + 2, *p_full = s_full + 2, *o_done = p_full + 2, *last_done = o_done + 2;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = (int)a.Hkv, G = pl.G;
  const int R = (int)(a.B * a.L) * G;
  const int64_t rows_out = a.B * a.L * a.H;

  if (threadIdx.x == 0) {
    mbar_init(last_done, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_free[s], 1);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_free[s], 1);
    }
    for (int s = 0; s < kSlots; ++s) mbar_init(&sc_full[s], 4);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 4);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_done[x], 1);
    }
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  griddep_wait();
  griddep_launch_dependents();

  Units un;
  un.tiles = pl.tc_tiles;
  un.u = (int)(blockIdx.x * pl.tc_units / pl.tc_ctas);
  un.end = (int)((blockIdx.x + 1) * pl.tc_units / pl.tc_ctas);
  int item, t0, n;

  if (warp < 8) {
    setmaxnreg_inc<kRegSoftmax>();
    const int x = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const uint32_t ts = tmem + lane_base + kColS + 128 * x, to = tmem + lane_base + kColO + 128 * x;
    int it = 0, sx = 0;  // tiles of the CTA, tiles of this row tile
    bool ok = true;
    while (ok && un.next(item, t0, n)) {
      const int j = item / pl.tc_groups;
      const int first = (item % pl.tc_groups) * kRowsCta + x * kRowsTile;
      if (first >= R) {  // no rows in tile B
        it += n;
        continue;
      }
      const int r = first + row;
      const int64_t out_row = r < R ? query_row(0, r, G, a.H, j) : 0;
      {  // the row's query in the operand's order
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + out_row * kD);
        uint8_t *dst = sm + kOffQ + x * kOperand + row * 128;
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < R) v = __ldg(src + c);
          *reinterpret_cast<uint4 *>(dst + (c >> 3) * (kOperand / 2) + (((c & 7) ^ (row & 7)) << 4)) =
              make_uint4(prmt(v.x, v.y, 0x5410), prmt(v.z, v.w, 0x5410), prmt(v.x, v.y, 0x7632),
                         prmt(v.z, v.w, 0x7632));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[x]);

      float m = 0.0f, shift = 0.0f, sum0 = 0.0f, sum1 = 0.0f;
      int e = kMinExp;
      for (int i = 0; i < n; ++i, ++it, ++sx) {
        const int slot = it & (kSlots - 1);
        const float *ks = scales + slot * 2 * kTokens, *vs = ks + kTokens;
        // the scores first: a tile that skipped row groups is then no further
        // than one phase from the scales' barrier, which has no count of its own
        ok = mbar_wait_warp(&s_full[x], sx & 1) && mbar_wait_warp(&sc_full[slot], (it / kSlots) & 1);
        if (!ok) break;
        tc_fence_after();
        float t[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) ld32(ts + 32 * c, t + 32 * c);
        tmem_ld_wait();
        float tm = -INFINITY, tn = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          const float4 k4 = *reinterpret_cast<const float4 *>(ks + c);
          f32x2_mul(t[c], t[c + 1], t[c], t[c + 1], k4.x, k4.y);
          f32x2_mul(t[c + 2], t[c + 3], t[c + 2], t[c + 3], k4.z, k4.w);
        }
        const int64_t left = a.P - (int64_t)(t0 + i) * kTokens;
        if (left < kTokens) {  // the prefix ends inside the tile
#pragma unroll
          for (int c = 0; c < 128; ++c) t[c] = c < left ? t[c] : -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          tm = max3(tm, t[c], t[c + 1]);
          tn = max3(tn, t[c + 2], t[c + 3]);
        }
        tm = fmaxf(tm, tn);
        const int4 e4 = *reinterpret_cast<const int4 *>(exps + 4 * slot);
        const int e_new = max(max(e, max(e4.x, e4.y)), max(e4.z, e4.w));
        if (i == 0) {
          m = tm;
          e = e_new;
          shift = m + (float)(e - kHead);
        } else if (__any_sync(0xffffffffu, tm > m + kSlack || e_new > e)) {
          if (tm > m + kSlack) m = tm;
          e = e_new;
          const float s_new = m + (float)(e - kHead);
          const float f = exp2_approx(shift - s_new);
          shift = s_new;
          sum0 *= f;
          sum1 *= f;
          ok = mbar_wait_warp(&o_done[x], (sx - 1) & 1);  // the output so far is complete
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            ld32(to + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= f;
            st32(to + 32 * c, o);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float *p = t + 32 * c + k;
            f32x2_sub(p[0], p[1], p[0], p[1], shift, shift);
            f32x2_sub(p[2], p[3], p[2], p[3], shift, shift);
#pragma unroll
            for (int q = 0; q < 4; ++q) p[q] = exp2_approx(p[q]);
            f32x2_add(sum0, sum1, sum0, sum1, p[0], p[1]);
            f32x2_add(sum0, sum1, sum0, sum1, p[2], p[3]);
            const float4 v4 = *reinterpret_cast<const float4 *>(vs + 32 * c + k);
            f32x2_mul(p[0], p[1], p[0], p[1], v4.x, v4.y);
            f32x2_mul(p[2], p[3], p[2], p[3], v4.z, v4.w);
            pk[k / 2] = pack_half2(p[0], p[1]);
            pk[k / 2 + 1] = pack_half2(p[2], p[3]);
          }
          tmem_st16(ts + 16 * c, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      ok = mbar_wait_warp(&o_done[x], (sx - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const float sum = sum0 + sum1, inv = 1.0f / sum;
      const int64_t at = (blockIdx.x - tc_cta_of(pl, (int64_t)item * pl.tc_tiles)) * rows_out + out_row;
      if (r < R) part_lse[at] = shift + log2f(sum);
      float4 *dst = reinterpret_cast<float4 *>(part_o + at * kD);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[32];
        ld32(to + 32 * c, o);
        tmem_ld_wait();
        if (r < R)
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            const float *p = o + k;
            dst[8 * c + k / 4] = make_float4(p[0] * inv, p[4] * inv, p[1] * inv, p[5] * inv);
            dst[8 * c + k / 4 + 1] = make_float4(p[2] * inv, p[6] * inv, p[3] * inv, p[7] * inv);
          }
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    setmaxnreg_dec<kRegOperand>();
    const int tid = threadIdx.x - 256, w = warp - 8;
    int it = 0;
    bool ok = true;
    Words kw, vw;
    bool more = un.next(item, t0, n);
    if (more)
      load_words<MODE>(kw, a.prefix.k_hi, a.prefix.k_lo, (int64_t)t0 * kTokens, a.P, Hkv,
                       item / pl.tc_groups, tid);
    while (ok && more) {
      const int j = item / pl.tc_groups;
      int next_item = item;
      int next_t0 = t0, next_n = n;
      for (int i = 0; i < n; ++i, ++it) {
        const int64_t tok = (int64_t)(t0 + i) * kTokens;
        const int s = it & (kStages - 1), slot = it & (kSlots - 1);
        const uint32_t free_parity = ((it / kStages) & 1) ^ 1;
        load_words<MODE>(vw, a.prefix.v_hi, a.prefix.v_lo, tok, a.P, Hkv, j, tid);
        float fk = 0.0f, fv = 0.0f;
        if (tok + tid < a.P) {
          const int64_t row = (tok + tid) * Hkv + j;
          fk = half_bits(__ldg(a.prefix.k_scale + row)) * (MODE ? 0.0625f * kScale : kScale);
          fv = half_bits(__ldg(a.prefix.v_scale + row)) * (MODE ? 0.0625f : 1.0f);
        }
        ok = mbar_wait_warp(&k_free[s], free_parity);
        if (!ok) break;
        scales[slot * 2 * kTokens + tid] = fk;
        scales[slot * 2 * kTokens + kTokens + tid] = fv;
        int e = fv > 0.0f ? (int)((__float_as_uint(fv) >> 23) & 0xFFu) - 126 : kMinExp;
        e = __reduce_max_sync(0xffffffffu, min(e, 40));
        if (lane == 0) exps[4 * slot + w] = e;
        store_words<MODE>(sm + kOffK + s * kOperand, kw, tid);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sc_full[slot]);
          mbar_arrive(&k_full[s]);
        }
        // the next tile's K words while V is written
        if (i + 1 < n) {
          load_words<MODE>(kw, a.prefix.k_hi, a.prefix.k_lo, tok + kTokens, a.P, Hkv, j, tid);
        } else {
          more = un.next(next_item, next_t0, next_n);
          if (more)
            load_words<MODE>(kw, a.prefix.k_hi, a.prefix.k_lo, (int64_t)next_t0 * kTokens, a.P, Hkv,
                             next_item / pl.tc_groups, tid);
        }
        ok = mbar_wait_warp(&v_free[s], free_parity);
        if (!ok) break;
        store_words<MODE>(sm + kOffV + s * kOperand, vw, tid);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[s]);
      }
      item = next_item;
      t0 = next_t0;
      n = next_n;
    }
  } else {
    setmaxnreg_dec<kRegIssue>();
    if (warp == 12 && lane == 0) {
      const uint64_t qd = umma_desc_sw128(sm + kOffQ), kd = umma_desc_sw128(sm + kOffK),
                     vd = desc_mn_sw128(sm + kOffV);
      constexpr uint64_t kOp = kOperand >> 4;  // descriptor address unit: 16 bytes
      int it = 0, seg = 0, seg_b = 0, sx[2] = {0, 0};
      bool ok = true, issued = false;
      auto scores = [&](int x, int s) {  // S_x = Q_x K^T: 8 k-steps of 16 columns
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t step = (k >> 2) * (kOp / 2) + 2 * (k & 3);
          mma_ss(tmem + kColS + 128 * x, qd + x * kOp + step, kd + s * kOp + step, idesc(false),
                 k > 0);
        }
        umma_commit(&s_full[x]);
        issued = true;
      };
      auto output = [&](int x, int s, bool add) {  // O_x += P_x V: 8 k-steps of 16 tokens
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ts(tmem + kColO + 128 * x, tmem + kColS + 128 * x + 8 * k,
                 vd + s * kOp + (2048 >> 4) * k, idesc(true), add || k > 0);
        umma_commit(&o_done[x]);
      };
      while (ok && un.next(item, t0, n)) {
        const bool two = (item % pl.tc_groups) * kRowsCta + kRowsTile < R;
        ok = mbar_wait(&q_full[0], seg & 1) && (!two || mbar_wait(&q_full[1], seg_b & 1)) &&
             mbar_wait(&k_full[it & 1], (it >> 1) & 1);
        if (!ok) break;
        ++seg;
        seg_b += two;
        tc_fence_after();
        scores(0, it & 1);
        if (two) scores(1, it & 1);
        umma_commit(&k_free[it & 1]);
        for (int i = 0; i < n; ++i, ++it) {
          const int s = it & 1, s2 = (it + 1) & 1;
          const uint32_t ph = (it >> 1) & 1, ph2 = ((it + 1) >> 1) & 1;
          const bool last = i + 1 == n;
          ok = mbar_wait(&v_full[s], ph) && mbar_wait(&p_full[0], sx[0] & 1);
          if (!ok) break;
          tc_fence_after();
          output(0, s, i > 0);
          ++sx[0];
          if (!last) {
            ok = mbar_wait(&k_full[s2], ph2);
            if (!ok) break;
            tc_fence_after();
            scores(0, s2);
          }
          if (two) {
            ok = mbar_wait(&p_full[1], sx[1] & 1);
            if (!ok) break;
            tc_fence_after();
            output(1, s, i > 0);
            ++sx[1];
          }
          umma_commit(&v_free[s]);
          if (!last) {
            if (two) scores(1, s2);
            umma_commit(&k_free[s2]);
          }
        }
      }
      // what was issued must end before tensor memory and the barriers go
      if (issued) {
        umma_commit(last_done);
        mbar_wait_final(last_done, 0);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_prefix_tc(const PrefixAttnArgs &a, const Plan &p, float *part_lse,
                             float *part_o, cudaStream_t st) {
  auto kern = a.mode ? prefix_tc_kernel<1> : prefix_tc_kernel<0>;
  // the register split hands out the launch allocation: not launched otherwise
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)p.tc_ctas), dim3(kThreads), kSmem, st, true, a, p,
                    part_lse, part_o);
}

}  // namespace pattn

cudaError_t read_wait_timeout_prefix(int *flag, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_wait_timeout, sizeof(int));
  if (e != cudaSuccess || !reset) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_wait_timeout, &zero, sizeof(int));
}

}  // namespace bitnest
