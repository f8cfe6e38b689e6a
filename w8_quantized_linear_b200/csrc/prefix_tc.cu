// Attention over a shared prefix on tcgen05, for the many rows (queries x
// heads of one KV head) that a batch gives: S = Q K^T and O = P V with 128 x
// 128 tiles, both accumulators in tensor memory, one pass with a running
// maximum.
//
// A CTA takes 256 rows of one KV head (two tiles, A and B; only A where there
// is little to do) and 128 tokens at a
// time, and an equal run of such units over all KV heads and row groups.  25
// warps:
//   0-15   softmax of tile A (0-7) and B (8-15), 16 rows a warp, four threads a
//          row (so that a token's scales serve two rows of a thread, and a
//          thread needs a quarter of them): the scores from tensor memory,
//          times the tokens' K scales, the row's running maximum,
//          p = 2^(s - shift), times the V scales, written back over the
//          scores as the second product's A operand, in two fp16 terms;
//   16-23  the cache's codes as fp16 operands: plane words -> shared memory
//          (128-byte swizzle), two stages of K and of V; the tokens' scales;
//   24     issues the MMAs.
// The tensor cores work on tile B while A is in its softmax and back; scores are
// computed a token tile ahead, in halves of 64 tokens, each into the place of the
// weights that the output before has used up.
//
// Measured: 128 x 4 queries of 32 heads over 16384 target tokens (8192 units, 56 a
// CTA) 235 us with the join, 585 TFLOP/s.  Under the profiler (252 us) a unit takes
// 7470 cycles: its MMAs need 3072, its exponentials 2048 (16 a cycle and SM), and no
// unit is full: the SM's load/store pipe, which tensor memory reads and writes, scales
// and operands share, 69 %, issue slots 52 %, tensor cores 41 %.  Without the second
// terms' MMAs it is 3 % faster: what bounds it is the chain from scores to weights to
// output of each half tile.
// Scores held in registers for both passes by fewer warps were slower.
//
// The codes are exact in fp16, so a score is off by fp32 sums only.  The
// output is rescaled only when a row's maximum has grown by 2^8 or the largest
// V scale has (the softmax warps do it in place): p is kept as 2^(s - shift)
// with shift = m + e - 7, m a maximum that is at most 8 behind, 2^e above every
// V scale so far, so p v_scale < 2^15 in fp16, with 2^29 between it and fp16's
// subnormals; row sums carry the same factor, which cancels.  p v_scale enters the
// product as two fp16 terms, 22 bits together: one alone would put 2^-11 of every
// weight into outputs that cancel.
//
// Columns of a head are kept in the order 0 2 4 6 1 3 5 7 within each 8 (the
// order in which plane words unpack with the fewest instructions): the same
// for Q and K, and undone when the output is written.
#include <math.h>

#include "nested_mma.cuh"
#include "prefix_plan.h"
#include "sm100.cuh"
#include "tc_f16.cuh"

namespace bitnest {
namespace pattn {

namespace {

using namespace nested;
using namespace tc16;

constexpr int kRowsTile = kTcTile, kTokens = kTcTokens;
constexpr int kSoftmaxWarps = 16, kOperandWarps = 8;
constexpr int kWords = 16 / kOperandWarps;  // rows of a tile for an operand thread
constexpr int kIssueWarp = kSoftmaxWarps + kOperandWarps;
constexpr int kThreads = (kSoftmaxWarps + kOperandWarps + 1) * 32;
constexpr int kStages = 2, kSlots = 4;
constexpr int kHalf = kTokens / 2;
constexpr int kOperand = kTokens * kD * 2;  // bytes of a K, V or Q tile
constexpr float kScale = 0.088388347648318440550f * 1.4426950408889634f;  // log2(e) / sqrt(128)
constexpr float kSlack = 8.0f;
constexpr int kHead = 7;  // p v_scale < 2^(8 + 7)
constexpr int kMinExp = -40;  // below any fp16 scale / 16

constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 2 * kOperand;
constexpr int kOffV = kOffK + kStages * kOperand;
// A slot's scales: token 8 n + 2 q + i at q * kScaleRow + 2 n + i, the order in which a
// softmax thread holds its columns (its lane % 4 = q), rows in different banks
constexpr int kScaleRow = 36, kScaleSet = 4 * kScaleRow;
constexpr int kOffScale = kOffV + kStages * kOperand;        // [slot][k, v][kScaleSet] floats
constexpr int kOffExp = kOffScale + kSlots * 2 * kScaleSet * 4;  // [slot][4] ints
constexpr int kOffBar = kOffExp + kSlots * 4 * 4;
constexpr int kBars = 4 * kStages + kSlots + 2 + 4 + 4 + 2 + 2 + 1;
constexpr int kSmem = kOffBar + kBars * 8 + 16 + 1024;

constexpr int kColO = 0, kColS = 256;  // tensor memory columns (tile B: + 128)

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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One operand thread's share of a tile's plane rows: for q < kWords, 16 bytes
// (piece tid / 8 % 4) of the row of token 8 kOperandWarps q + 8 (tid / 32) + tid % 8.
constexpr int kRowStep = 8 * kOperandWarps;
struct Words {
  uint4 hi[kWords], lo[kWords];
};
struct Rows {  // where a thread's rows of a tile are
  int64_t t, off;
};
__device__ __forceinline__ Rows rows_of(int64_t t0, int64_t Hkv, int j, int tid) {
  const int64_t t = t0 + 8 * (tid >> 5) + (tid & 7);
  return {t, (t * Hkv + j) * (kD / 2) + 16 * ((tid >> 3) & 3)};
}
template <int MODE>
__device__ __forceinline__ void load_words(Words &w, int q, const uint8_t *__restrict__ hi,
                                           const uint8_t *__restrict__ lo, const Rows &r,
                                           int64_t P, int64_t Hkv) {
  w.hi[q] = w.lo[q] = make_uint4(0, 0, 0, 0);
  if (r.t + kRowStep * q < P) {
    const int64_t off = r.off + q * kRowStep * Hkv * (kD / 2);
    w.hi[q] = __ldg(reinterpret_cast<const uint4 *>(hi + off));
    if (MODE) w.lo[q] = __ldg(reinterpret_cast<const uint4 *>(lo + off));
  }
}
// ... as fp16 to the tile at `dst`: token rows of 128 bytes in two halves (64
// columns each, 16 KB apart), 16-byte chunk c of row t at c ^ (t % 8).  The
// eight lanes of a store phase have tokens of different t % 8: different banks.
template <int MODE>
__device__ __forceinline__ void store_words(uint8_t *dst, const Words &w, int q, int tid) {
  const int piece = (tid >> 3) & 3, t = 8 * (tid >> 5) + (tid & 7);
  uint8_t *row = dst + (piece >> 1) * (kOperand / 2) + (t + kRowStep * q) * 128;
  const uint32_t h[4] = {w.hi[q].x, w.hi[q].y, w.hi[q].z, w.hi[q].w};
  const uint32_t l[4] = {w.lo[q].x, w.lo[q].y, w.lo[q].z, w.lo[q].w};
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4 *>(row + ((((piece & 1) * 4 + c) ^ (t & 7)) << 4)) =
        codes8<MODE>(h[c], l[c]);
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
  uint8_t *sm = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an integer cast would lose the address space)
  float *scales = reinterpret_cast<float *>(sm + kOffScale);
  int *exps = reinterpret_cast<int *>(sm + kOffExp);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kOffBar);
  uint64_t *k_full = bars, *k_free = k_full + kStages, *v_full = k_free + kStages,
           *v_free = v_full + kStages, *sc_full = v_free + kStages, *q_full = sc_full + kSlots,
           *s_full = q_full + 2, *p_full = s_full + 4, *o_done = p_full + 4, *o_last = o_done + 2, *last_done = o_last + 2;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = (int)a.Hkv, lgG = pl.lgG;
  const int R = (int)(a.B * a.L) << lgG;
  const int64_t rows_out = a.B * a.L * a.H;

  if (threadIdx.x == 0) {
    mbar_init(last_done, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], kOperandWarps);
      mbar_init(&k_free[s], 1);
      mbar_init(&v_full[s], kOperandWarps);
      mbar_init(&v_free[s], 1);
    }
    for (int s = 0; s < kSlots; ++s) mbar_init(&sc_full[s], 4);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], kSoftmaxWarps / 2);
      mbar_init(&o_done[x], 1);
      mbar_init(&o_last[x], 1);
    }
    for (int x = 0; x < 4; ++x) {  // [row tile][half of the token tile]
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], kSoftmaxWarps / 2);
    }
    fence_barrier_init();
  }
  if (warp == kIssueWarp) {
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
  un.u = blockIdx.x * pl.tc_run;
  un.end = min(un.u + pl.tc_run, pl.tc_units);
  int item, t0, n;

  if (warp < kSoftmaxWarps) {
    // tile x; rows 32 (warp % 4) + 16 (warp / 4 % 2) .. + 15 of it, this
    // thread's: lane / 4 and lane / 4 + 8 of those
    const int x = warp >> 3, first_row = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
    const uint32_t ts = tmem + ((uint32_t)first_row << 16) + kColS + 128 * x,
                   to = tmem + ((uint32_t)first_row << 16) + kColO + 128 * x;
    int it = 0, su = 0, groups = 0;  // token tiles of the CTA, half tiles and row groups of this row tile
    bool ok = true;
    while (ok && un.next(item, t0, n)) {
      const int j = item / pl.tc_groups;
      const int first = (item % pl.tc_groups) * pl.tc_rows + x * kRowsTile;
      if (first >= R || x * kRowsTile >= pl.tc_rows) {  // no rows in tile B
        it += n;
        continue;
      }
      {  // half of a row's query for each thread, in the operand's order
        const int row = first_row + (lane >> 1), r = first + row, half = lane & 1;
        const uint4 *src = reinterpret_cast<const uint4 *>(
                               a.q + (r < R ? query_row(0, r, lgG, (int)a.H, j) : 0) * kD) + 8 * half;
        uint8_t *dst = sm + kOffQ + x * kOperand + half * (kOperand / 2) + row * 128;
#pragma unroll 4
        for (int c = 0; c < 8; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < R) v = __ldg(src + c);
          *reinterpret_cast<uint4 *>(dst + ((c ^ (row & 7)) << 4)) =
              make_uint4(prmt(v.x, v.y, 0x5410), prmt(v.z, v.w, 0x5410), prmt(v.x, v.y, 0x7632),
                         prmt(v.z, v.w, 0x7632));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[x]);

      float m[2], shift[2], sum[2][2];
      int e = kMinExp;
#pragma unroll
      for (int r = 0; r < 2; ++r) m[r] = shift[r] = sum[r][0] = sum[r][1] = 0.0f;
      for (int i = 0; i < 2 * n; ++i, ++su) {
        const int half = i & 1, slot = (it + (i >> 1)) & (kSlots - 1);
        const uint32_t th = ts + kHalf * half;
        const float *ks = scales + slot * 2 * kScaleSet + (lane & 3) * kScaleRow + 16 * half, *vs = ks + kScaleSet;
        // the scores first: a tile that skipped row groups is then no further
        // than one phase from the scales' barrier, which has no count of its own
        ok = wait_warp(&s_full[2 * x + half], (su >> 1) & 1) &&
             wait_warp(&sc_full[slot], ((it + (i >> 1)) / kSlots) & 1);
        if (!ok) break;
        tc_fence_after();
        float t[32], tm[2] = {-INFINITY, -INFINITY};
        ld_16x64(th, t);
        ld_wait32(t);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 k4 = *reinterpret_cast<const float4 *>(ks + 4 * k);
          float *p = t + 8 * k;
          f32x2_mul(p[0], p[1], p[0], p[1], k4.x, k4.y);
          f32x2_mul(p[2], p[3], p[2], p[3], k4.x, k4.y);
          f32x2_mul(p[4], p[5], p[4], p[5], k4.z, k4.w);
          f32x2_mul(p[6], p[7], p[6], p[7], k4.z, k4.w);
        }
        const int left = (int)a.P - (t0 + (i >> 1)) * kTokens - kHalf * half;
        if (left < kHalf) {  // the prefix ends inside the half tile, or before it
#pragma unroll
          for (int k = 0; k < 32; ++k)
            t[k] = 8 * (k >> 2) + 2 * (lane & 3) + (k & 1) < left ? t[k] : -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          tm[0] = max3(tm[0], t[k], t[k + 1]);
          tm[1] = max3(tm[1], t[k + 2], t[k + 3]);
        }
        const int4 e4 = *reinterpret_cast<const int4 *>(exps + 4 * slot);
        const int e_new = max(max(e, max(e4.x, e4.y)), max(e4.z, e4.w));
        bool grown = e_new > e;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          tm[r] = fmaxf(tm[r], __shfl_xor_sync(0xffffffffu, tm[r], 1));
          tm[r] = fmaxf(tm[r], __shfl_xor_sync(0xffffffffu, tm[r], 2));
          grown |= tm[r] > m[r] + kSlack;
        }
        if (i == 0) {
          e = e_new;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            m[r] = tm[r];
            shift[r] = m[r] + (float)(e - kHead);
          }
        } else if (__any_sync(0xffffffffu, grown)) {
          e = e_new;
          float f[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (tm[r] > m[r] + kSlack) m[r] = tm[r];
            const float s_new = m[r] + (float)(e - kHead);
            f[r] = exp2_approx(shift[r] - s_new);
            shift[r] = s_new;
            sum[r][0] *= f[r];
            sum[r][1] *= f[r];
          }
          ok = wait_warp(&o_done[x], (su - 1) & 1);  // the output so far is complete
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kD / 8; ++c) {
            float o[4];
            ld_16x8(to + 8 * c, o);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] *= f[k >> 1];
            st_16x8(to + 8 * c, o);
          }
        }
        uint32_t pk[16], pl[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float *p = t + 8 * k;
          const float4 v4 = *reinterpret_cast<const float4 *>(vs + 4 * k);
#pragma unroll
          for (int q = 0; q < 8; q += 2) {  // row lane / 4 + 8 (q / 2 % 2), two tokens
            const int r = (q >> 1) & 1;
            f32x2_sub(p[q], p[q + 1], p[q], p[q + 1], shift[r], shift[r]);
            p[q] = exp2_approx(p[q]);
            p[q + 1] = exp2_approx(p[q + 1]);
            f32x2_add(sum[r][0], sum[r][1], sum[r][0], sum[r][1], p[q], p[q + 1]);
            f32x2_mul(p[q], p[q + 1], p[q], p[q + 1], q < 4 ? v4.x : v4.z, q < 4 ? v4.y : v4.w);
            pk[4 * k + q / 2] = split_half2(p[q], p[q + 1], pl[4 * k + q / 2]);
          }
        }
        // over the scores (all read): the first terms, the second ones behind them
        st_16x32(th, pk);
        st_16x32(th + kHalf / 2, pl);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + half]);
      }
      it += n;
      if (!ok) break;
      // All outputs of the row group, on a barrier that completes once a group: o_done
      // may be one or two phases on by now, and a wait for the parity of the first of
      // two that are both complete would wait for a third, which does not come.
      ok = wait_warp(&o_last[x], groups & 1);
      if (!ok) break;
      ++groups;
      tc_fence_after();
      const int64_t part = (int64_t)((int)blockIdx.x - tc_first_cta(pl, item)) * rows_out;
      float inv[2];
      float *dst[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float v = sum[r][0] + sum[r][1];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        inv[r] = 1.0f / v;
        const int row = first + first_row + (lane >> 2) + 8 * r;
        const int64_t at = part + (row < R ? query_row(0, row, lgG, (int)a.H, j) : 0);
        if (row < R && (lane & 3) == 0) part_lse[at] = shift[r] + log2f(v);
        // lane % 4 = 0 .. 3 writes columns 0, 4, 2, 6 and the one behind of each 8
        dst[r] = row < R ? part_o + at * kD + 4 * (lane & 1) + (lane & 2) : nullptr;
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float o[32];
        ld_16x64(to + 64 * g, o);
        ld_wait32(o);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const int r = (k >> 1) & 1;
          // this thread has two columns of equal parity, lane ^ 2 their neighbours
          const float give = (lane & 2) ? o[k] : o[k + 1];
          const float got = __shfl_xor_sync(0xffffffffu, give, 2);
          const float2 w = (lane & 2) ? make_float2(got, o[k + 1]) : make_float2(o[k], got);
          if (dst[r])
            *reinterpret_cast<float2 *>(dst[r] + 64 * g + 8 * (k >> 2)) =
                make_float2(w.x * inv[r], w.y * inv[r]);
        }
      }
      tc_fence_before();
    }
  } else if (warp < kIssueWarp) {
    const int tid = threadIdx.x - 32 * kSoftmaxWarps, w = warp - kSoftmaxWarps;
    const KvPlanes &c = a.prefix;
    // The CTA's token tiles one after the other, across row groups: K of the
    // next tile, then V of this one.  Each has words of its own in registers,
    // loaded as soon as the ones before are written: a load is in flight while
    // the other operand is written.
    const int tiles = un.end - un.u;
    struct Cursor {  // the tile to load next
      Units un;
      int item, t, n;
      __device__ __forceinline__ void step() {
        ++t;
        if (--n == 0) un.next(item, t, n);
      }
    } ck, cv;
    ck.un = un;
    ck.un.next(ck.item, ck.t, ck.n);
    cv = ck;
    Words kw, vw;
    uint16_t sk = 0, sv = 0;
    auto load_k = [&]() {
      const int j = ck.item / pl.tc_groups;
      const Rows r = rows_of((int64_t)ck.t * kTokens, Hkv, j, tid);
#pragma unroll
      for (int q = 0; q < kWords; ++q) load_words<MODE>(kw, q, c.k_hi, c.k_lo, r, a.P, Hkv);
      const int64_t tok = (int64_t)ck.t * kTokens + tid;
      sk = sv = 0;
      if (w < 4 && tok < a.P) {
        sk = __ldg(c.k_scale + tok * Hkv + j);
        sv = __ldg(c.v_scale + tok * Hkv + j);
      }
      ck.step();
    };
    auto load_v = [&]() {
      const Rows r = rows_of((int64_t)cv.t * kTokens, Hkv, cv.item / pl.tc_groups, tid);
#pragma unroll
      for (int q = 0; q < kWords; ++q) load_words<MODE>(vw, q, c.v_hi, c.v_lo, r, a.P, Hkv);
      cv.step();
    };
    auto store_k = [&](int it) {
      const int s = it & (kStages - 1), slot = it & (kSlots - 1);
      if (!wait_warp(&k_free[s], ((it / kStages) & 1) ^ 1)) return false;
      if (w < 4) {  // a token's scales for each of 128 threads
        const float fk = half_bits(sk) * (MODE ? 0.0625f * kScale : kScale);
        const float fv = half_bits(sv) * (MODE ? 0.0625f : 1.0f);
        const int sc = slot * 2 * kScaleSet + ((tid >> 1) & 3) * kScaleRow + 2 * (tid >> 3) + (tid & 1);
        scales[sc] = fk;
        scales[sc + kScaleSet] = fv;
        int e = fv > 0.0f ? (int)((__float_as_uint(fv) >> 23) & 0xFFu) - 126 : kMinExp;
        e = __reduce_max_sync(0xffffffffu, min(e, 40));
        if (lane == 0) exps[4 * slot + w] = e;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[slot]);
      }
#pragma unroll
      for (int q = 0; q < kWords; ++q) store_words<MODE>(sm + kOffK + s * kOperand, kw, q, tid);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[s]);
      if (it + 1 < tiles) load_k();
      return true;
    };
    bool ok = true;
    if (tiles > 0) {
      load_k();
      load_v();
      ok = store_k(0) && (tiles == 1 || store_k(1));
    }
    for (int it = 0; ok && it < tiles; ++it) {
      const int s = it & (kStages - 1);
      ok = wait_warp(&v_free[s], ((it / kStages) & 1) ^ 1);
      if (!ok) break;
#pragma unroll
      for (int q = 0; q < kWords; ++q) store_words<MODE>(sm + kOffV + s * kOperand, vw, q, tid);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[s]);
      if (it + 1 < tiles) load_v();
      if (it + 2 < tiles) ok = store_k(it + 2);
    }
  } else {
    {
      const uint64_t qd = umma_desc_sw128(sm + kOffQ), kd = umma_desc_sw128(sm + kOffK),
                     vd = desc_mn_sw128(sm + kOffV);
      constexpr uint64_t kOp = kOperand >> 4;  // descriptor address unit: 16 bytes
      int it = 0, seg = 0, seg_b = 0, su[2] = {0, 0};
      bool ok = true, issued = false;
      // The whole warp runs along and one elected thread issues.
      // S_x = Q_x K^T for a half of the token tile in stage s: 8 k-steps of 16 columns
      auto scores = [&](int x, int s, int half) {
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint64_t step = (k >> 2) * (kOp / 2) + 2 * (k & 3);
            mma_ss(tmem + kColS + 128 * x + kHalf * half, qd + x * kOp + step,
                   kd + s * kOp + half * (kHalf * 128 >> 4) + step, idesc(false, kHalf), k > 0);
          }
          umma_commit(&s_full[2 * x + half]);
        }
        __syncwarp();
        issued = true;
      };
      // O_x += P_x V for a half: 4 k-steps of 16 tokens of each of the weights' two terms
      auto output = [&](int x, int s, int half, bool add) {
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts(tmem + kColO + 128 * x, tmem + kColS + 128 * x + kHalf * half + 8 * k,
                   vd + s * kOp + (2048 >> 4) * (4 * half + (k & 3)), idesc(true, kD), add || k > 0);
          umma_commit(&o_done[x]);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t *bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      while (ok && un.next(item, t0, n)) {
        const bool two = pl.tc_rows > kRowsTile && (item % pl.tc_groups) * pl.tc_rows + kRowsTile < R;
        ok = wait_warp(&q_full[0], seg & 1) && (!two || wait_warp(&q_full[1], seg_b & 1)) &&
             wait_warp(&k_full[it & 1], (it >> 1) & 1);
        if (!ok) break;
        ++seg;
        seg_b += two;
        tc_fence_after();
        for (int half = 0; half < 2; ++half) {
          scores(0, it & 1, half);
          if (two) scores(1, it & 1, half);
        }
        commit(&k_free[it & 1]);
        // Scores are a token tile ahead: each half's are computed into the place of
        // the weights that its output has just used up.
        for (int i = 0; i < n; ++i, ++it) {
          const int s = it & 1, s2 = (it + 1) & 1;
          const bool last = i + 1 == n;
          ok = wait_warp(&v_full[s], (it >> 1) & 1) && (last || wait_warp(&k_full[s2], ((it + 1) >> 1) & 1));
          if (!ok) break;
          for (int half = 0; ok && half < 2; ++half) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (x == 1 && !two) break;
              ok = ok && wait_warp(&p_full[2 * x + half], (su[x] >> 1) & 1);
              if (!ok) break;
              tc_fence_after();
              output(x, s, half, i > 0 || half > 0);
              if (last && half == 1) commit(&o_last[x]);
              ++su[x];
            }
            // products into different columns are not bound to run in order: the scores
            // wait for the output that still reads the weights in their place
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (last || (x == 1 && !two)) break;
              ok = ok && wait_warp(&o_done[x], (su[x] - 1) & 1);
              if (!ok) break;
              tc_fence_after();
              scores(x, s2, half);
            }
          }
          if (!ok) break;
          commit(&v_free[s]);
          if (!last) commit(&k_free[s2]);
        }
      }
      // what was issued must end before tensor memory and the barriers go
      if (issued) {
        commit(last_done);
        mbar_wait_final(last_done, 0);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_prefix_tc(const PrefixAttnArgs &a, const Plan &p, float *part_lse,
                             float *part_o, cudaStream_t st) {
  auto kern = a.mode ? prefix_tc_kernel<1> : prefix_tc_kernel<0>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
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
