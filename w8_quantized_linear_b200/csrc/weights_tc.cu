// The attention weight that a shared prefix's tokens received, on tcgen05, for
// the many rows (queries x heads of one KV head) of a batch:
//   acc[t] += sum_r exp(q_r k_t / sqrt(128) - lse_r).
// Tokens are the products' rows: S = K Q^T with 128 tokens x 128 rows, so a
// token's sum stays in one quarter-warp for the whole pass, and nothing is
// reduced across threads before the end.
//
// A CTA takes an equal run of token tiles over all KV heads, two at a time (a
// segment), whose codes stay in shared memory while the rows pass by in tiles
// of 128.  Four slots (128 columns of tensor memory, four warps) work at a
// time, on two row tiles of each of two token tiles, or on four of one.  The
// next segment's codes are written meanwhile.  22 warps:
//   0-15   slot warp / 4: the weights of its products from tensor memory, in
//          pieces of 16 tokens x 64 rows;
//   16-19  codes -> fp16 operand, and the tokens' scales;
//   20     issues the MMAs;
//   21     brings the row tiles (TMA) and their lse.
//
// The exponentials, 16 a cycle and SM, make 1024 cycles a product of 128 x 128, its
// MMAs 512.  64 x 4 queries of 32 heads over 16384 tokens: 50 us, 689 TFLOP/s, of
// which the exponentials are 31 at least (their unit is busy 63 % of the time); a
// quarter of them as polynomials on the FMA pipe instead takes 52: what is left is
// the reading of tensor memory and the slots' hand-over.
#include <cudaTypedefs.h>
#include <math.h>

#include "launch.h"
#include "nested_mma.cuh"
#include "sm100.cuh"
#include "tc_f16.cuh"

namespace bitnest {
namespace evict {

namespace {

using namespace nested;
using namespace tc16;

constexpr int kSms = 148;
constexpr int kTile = 128;
constexpr int kSlots = 4, kPair = 2, kStages = 2, kSets = 16;
constexpr int kSlotWarps = 4 * kSlots, kCodeWarps = 4;
constexpr int kIssueWarp = kSlotWarps + kCodeWarps, kRowWarp = kIssueWarp + 1;
constexpr int kThreads = (kRowWarp + 1) * 32;
constexpr int kOperand = kTile * kD * 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kScale = 0.088388347648318440550f * kLog2e;  // log2(e) / sqrt(128)

// A set: -lse log2(e) of a row tile, row 8 n + 2 q + i at q * kSetRow + 2 n + i, the
// order in which a thread of lane % 4 = q holds its columns, rows in different banks.
// The loader writes row tile i's set when the stage of row tile i - kStages is free,
// that is, when that tile's products are issued.  A slot has read a set when its next
// product is issued, which is at most 2 kSlots - 1 row tiles later: where a segment of
// one token tile has 4 n + 3 row tiles, its last round leaves out slot 3, and in the
// next segment slot 3 comes fourth (a slot that a whole segment leaves out is bound by
// the barrier at the segment's end).
constexpr int kSetRow = 36, kSet = 4 * kSetRow;
static_assert(kSets - kStages >= 2 * kSlots - 1 && (kSets & (kSets - 1)) == 0, "a set is read before it is written");
constexpr int kOffK = 0;  // [segment % 2][tile]
constexpr int kOffQ = kOffK + 2 * kPair * kOperand;
constexpr int kOffSet = kOffQ + kStages * kOperand;
constexpr int kOffPart = kOffSet + kSets * kSet * 4;        // [segment % 2][slot][token]
constexpr int kOffFactor = kOffPart + 2 * kSlots * kTile * 4;  // [segment % 2][tile][token]
constexpr int kOffBar = kOffFactor + 2 * kPair * kTile * 4;
constexpr int kBars = 2 * kStages + kSets + 2 * kSlots + 4 + 1;
constexpr int kSmem = kOffBar + kBars * 8 + 16 + 1024;

__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, uint64_t *bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

struct Segment {  // token tiles first .. first + nt - 1 of KV head j
  int j, first, nt, ways;
};
struct Run {  // a CTA's run of tiles
  int u, end, per_head;
  __device__ __forceinline__ bool next(Segment &s) {
    if (u >= end) return false;
    s.j = u / per_head;
    s.first = u - s.j * per_head;
    s.nt = min(min(end - u, per_head - s.first), kPair);
    s.ways = kSlots / s.nt;
    u += s.nt;
    return true;
  }
};

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) weights_tc_kernel(
    const __grid_constant__ CUtensorMap tm_q, KvWeightsArgs a, int lgG) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + (-smem_u32(smem_raw) & 1023u);
  float *sets = reinterpret_cast<float *>(sm + kOffSet);
  float *part = reinterpret_cast<float *>(sm + kOffPart);
  float *factor = reinterpret_cast<float *>(sm + kOffFactor);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kOffBar);
  uint64_t *q_full = bars, *q_free = q_full + kStages, *set_full = q_free + kStages,
           *s_full = set_full + kSets, *s_free = s_full + kSlots, *k_full = s_free + kSlots,
           *k_free = k_full + 2, *last_done = k_free + 2;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = (int)a.Hkv, cap = (int)a.cap, G = 1 << lgG, R = (int)(a.B * a.L) << lgG;
  const int row_tiles = (R + kTile - 1) / kTile;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_free[s], 1);
    }
    for (int s = 0; s < kSets; ++s) mbar_init(&set_full[s], 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], kCodeWarps);
      mbar_init(&k_free[s], kSlotWarps + 1);
    }
    mbar_init(last_done, 1);
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

  Run run;
  run.per_head = (cap + kTile - 1) / kTile;
  const int64_t tiles = (int64_t)Hkv * run.per_head;
  run.u = (int)(blockIdx.x * tiles / gridDim.x);
  run.end = (int)((blockIdx.x + 1) * tiles / gridDim.x);
  Segment sg;

  if (warp < kSlotWarps) {
    const int slot = warp >> 2, quarter = warp & 3;
    const uint32_t ts = tmem + ((uint32_t)(32 * quarter) << 16) + kTile * slot;
    int uses = 0, q0 = 0;  // of this slot; row tiles before this segment
    bool ok = true;
    for (int seg = 0; run.next(sg); ++seg) {
      const int tile = slot % sg.nt, phase = slot / sg.nt, buf = seg & 1;
      const int t0 = (sg.first + tile) * kTile;
      // this thread's tokens: lane / 4 + 8 i of the warp's 32
      float f[4], sum[4][2];
      const int mine = t0 + 32 * quarter + lane;  // and the one whose sum it adds, if phase is 0
      float *const acc = a.acc + (int64_t)sg.j * cap + mine;
      const float old = phase == 0 && mine < cap ? *acc : 0.0f;  // early: used at the end
      ok = ok && wait_warp(&k_full[buf], (seg >> 1) & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = factor[(buf * kPair + tile) * kTile + 32 * quarter + 8 * i + (lane >> 2)];
        sum[i][0] = sum[i][1] = 0.0f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_free[buf]);
      for (int i = phase; ok && i < row_tiles; i += sg.ways) {
        const int set = (q0 + i) & (kSets - 1);
        const float *b = sets + set * kSet + (lane & 3) * kSetRow;
        ok = wait_warp(&s_full[slot], uses & 1) && wait_warp(&set_full[set], ((q0 + i) / kSets) & 1);
        if (!ok) break;
        ++uses;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float4 b4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) b4[k] = *reinterpret_cast<const float4 *>(b + 16 * g + 4 * k);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float t[32];
            ld_16x64(ts + ((uint32_t)h << 20) + 64 * g, t);
            ld_wait32(t);
            if (g == 1 && h == 1) {  // all read: the slot is free for the next product
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_free[slot]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int q = 0; q < 8; q += 2) {
                const int r = 2 * h + ((q >> 1) & 1);
                float *p = t + 8 * k + q;
                f32x2_fma(p[0], p[1], p[0], p[1], f[r], f[r], q < 4 ? b4[k].x : b4[k].z,
                          q < 4 ? b4[k].y : b4[k].w);
                p[0] = exp2_approx(p[0]);
                p[1] = exp2_approx(p[1]);
                f32x2_add(sum[r][0], sum[r][1], sum[r][0], sum[r][1], p[0], p[1]);
              }
          }
        }
      }
      q0 += row_tiles;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = sum[i][0] + sum[i][1];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if ((lane & 3) == 0)
          part[(buf * kSlots + slot) * kTile + 32 * quarter + 8 * i + (lane >> 2)] = v;
      }
      // every slot comes here, after a wait that gave up too
      asm volatile("bar.sync 1, %0;" ::"n"(kSlotWarps * 32) : "memory");
      if (phase == 0 && ok && mine < cap) {
        float v = 0.0f;
        for (int w = 0; w < sg.ways; ++w) v += part[(buf * kSlots + w * sg.nt + tile) * kTile + 32 * quarter + lane];
        *acc = old + v;
      }
      __syncwarp();
    }
  } else if (warp < kIssueWarp) {
    const int row = threadIdx.x - 32 * kSlotWarps;  // a thread's token of a tile
    bool ok = true;
    for (int seg = 0; ok && run.next(sg); ++seg) {
      const int buf = seg & 1;
      for (int tile = 0; tile < sg.nt; ++tile) {
        const int t = (sg.first + tile) * kTile + row;
        uint8_t *dst = sm + kOffK + (buf * kPair + tile) * kOperand + row * 128;
        const int64_t at = (int64_t)t * Hkv + sg.j, off = at * (kD / 2);
        uint4 hi[4], lo[4];
        float f = 0.0f;
#pragma unroll
        for (int p = 0; p < 4; ++p) hi[p] = lo[p] = make_uint4(0, 0, 0, 0);
        if (t < cap) {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            hi[p] = __ldg(reinterpret_cast<const uint4 *>(a.k_hi + off) + p);
            if (MODE) lo[p] = __ldg(reinterpret_cast<const uint4 *>(a.k_lo + off) + p);
          }
          f = half_bits(__ldg(a.k_scale + at)) * (MODE ? 0.0625f * kScale : kScale);
        }
        if (tile == 0) {
          ok = wait_warp(&k_free[buf], ((seg >> 1) & 1) ^ 1);
          if (!ok) break;
        }
        factor[(buf * kPair + tile) * kTile + row] = f;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t hw[4] = {hi[p].x, hi[p].y, hi[p].z, hi[p].w},
                         lw[4] = {lo[p].x, lo[p].y, lo[p].z, lo[p].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 8 columns
            uint32_t ev, od;
            codes<MODE>(hw[c], lw[c], ev, od);
            const int chunk = 4 * (p & 1) + c;
            *reinterpret_cast<uint4 *>(dst + (p >> 1) * (kOperand / 2) + ((chunk ^ (row & 7)) << 4)) =
                make_uint4(pair<MODE>(ev, od, 0), pair<MODE>(ev, od, 1), pair<MODE>(ev, od, 2),
                           pair<MODE>(ev, od, 3));
          }
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[buf]);
    }
  } else if (warp == kRowWarp) {
    int it = 0;  // row tiles of the CTA
    bool ok = true;
    while (ok && run.next(sg)) {
      for (int i = 0; i < row_tiles; ++i, ++it) {
        const int stage = it & (kStages - 1), set = it & (kSets - 1);
        ok = wait_warp(&q_free[stage], ((it / kStages) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {  // rows of zeros behind the last
          uint8_t *dst = sm + kOffQ + stage * kOperand;
          mbar_arrive_expect_tx(&q_full[stage], kOperand);
          tma_load_3d(dst, &tm_q, &q_full[stage], 0, sg.j * G, i * (kTile / G));
          tma_load_3d(dst + kOperand / 2, &tm_q, &q_full[stage], kD / 2, sg.j * G, i * (kTile / G));
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int c = 32 * n + lane, r = i * kTile + c;
          // a row without weight (lse -inf), or behind the last, gives none
          const float e = r < R ? __ldg(a.lse + query_row(0, r, lgG, (int)a.H, sg.j)) : -INFINITY;
          sets[set * kSet + ((c >> 1) & 3) * kSetRow + 2 * (c >> 3) + (c & 1)] =
              e == -INFINITY ? -INFINITY : -e * kLog2e;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&set_full[set]);
      }
    }
    if (!ok && lane == 0)  // gave up: let the copies already issued land
      for (int i = it > kStages ? it - kStages : 0; i < it; ++i)
        mbar_wait_final(&q_full[i & (kStages - 1)], (i / kStages) & 1);
    __syncwarp();
  } else {
    const uint64_t kd = umma_desc_sw128(sm + kOffK), qd = umma_desc_sw128(sm + kOffQ);
    constexpr uint64_t kOp = kOperand >> 4;  // descriptor address unit: 16 bytes
    int it0 = 0, uses[kSlots] = {};
    bool ok = true, issued = false;
    for (int seg = 0; ok && run.next(sg); ++seg) {
      const int buf = seg & 1;
      ok = wait_warp(&k_full[buf], (seg >> 1) & 1);
      for (int i0 = 0; ok && i0 < row_tiles; i0 += sg.ways) {
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
          const int phase = s / sg.nt, tile = s - phase * sg.nt, i = i0 + phase;
          if (!ok || i >= row_tiles) continue;
          const int stage = (it0 + i) & (kStages - 1);
          if (tile == 0) ok = wait_warp(&q_full[stage], ((it0 + i) / kStages) & 1);
          ok = ok && wait_warp(&s_free[s], (uses[s] & 1) ^ 1);
          if (!ok) continue;
          ++uses[s];
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint64_t step = (k >> 2) * (kOp / 2) + 2 * (k & 3);
              mma_ss(tmem + kTile * s, kd + (buf * kPair + tile) * kOp + step,
                     qd + stage * kOp + step, idesc(false), k > 0);
            }
            umma_commit(&s_full[s]);
            if (tile == sg.nt - 1) umma_commit(&q_free[stage]);
          }
          __syncwarp();
          issued = true;
        }
      }
      if (ok) {
        if (elect_one()) umma_commit(&k_free[buf]);
        __syncwarp();
      }
      it0 += row_tiles;
    }
    // what was issued must end before tensor memory and the barriers go
    if (issued) {
      if (elect_one()) umma_commit(last_done);
      __syncwarp();
      mbar_wait_final(last_done, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                        cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ok ? ptr : nullptr);
  }();
  return fn;
}

}  // namespace

cudaError_t launch_weights_tc(const KvWeightsArgs &a, cudaStream_t st) {
  const int64_t tiles = a.Hkv * ((a.cap + kTile - 1) / kTile);
  const int G = (int)(a.H / a.Hkv);
  int lgG = 0;
  while ((1 << lgG) < G) ++lgG;
  // q [B L, H, 128]: a row tile is 128 / G queries of one KV head's G heads, in
  // two halves of 64 columns
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  CUtensorMap tm;
  const cuuint64_t dims[3] = {kD, (cuuint64_t)a.H, (cuuint64_t)(a.B * a.L)};
  const cuuint64_t strides[2] = {2 * kD, (cuuint64_t)a.H * 2 * kD};
  const cuuint32_t box[3] = {kD / 2, (cuuint32_t)G, (cuuint32_t)(kTile / G)}, estr[3] = {1, 1, 1};
  if (fn(&tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t *>(a.q), dims, strides, box,
         estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  auto kern = a.mode ? weights_tc_kernel<1> : weights_tc_kernel<0>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)(tiles < kSms ? tiles : kSms)), dim3(kThreads), kSmem, st,
                    true, tm, a, lgG);
}

}  // namespace evict

cudaError_t read_wait_timeout_weights(int *flag, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_wait_timeout, sizeof(int));
  if (e != cudaSuccess || !reset) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_wait_timeout, &zero, sizeof(int));
}

}  // namespace bitnest
