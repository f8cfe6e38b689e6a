// A bounded nested KV cache: the attention weight each cached token has
// received, and eviction of the tokens that received least.
#include <algorithm>

#include "launch.h"
#include "nested_mma.cuh"
#include "sm100.cuh"

namespace bitnest {

namespace evict {

using namespace nested;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kScale = 0.088388347648318440550f * kLog2e;  // log2(e) / sqrt(128)

// ---------------------------------------------------------------- weights
// For more than 128 rows of one sequence's KV head and its own tokens (else
// few_rows_kernel below; a shared prefix of many rows: weights_tc.cu):
// acc[t] += sum over the rows (queries x heads of the KV head) that see token
// t of exp(q k_t / sqrt(128) - lse): the scores once more, from the K planes
// alone, with no maximum to keep since lse is known.  A warp holds the codes
// of 32 tokens as B operands for all rows; the rows pass by 16 at a time.  A
// token's sum is kept by the lanes that hold it, in a fixed order: no atomics.
constexpr int kWarps = 8;
constexpr int kTokens = 32;  // of a warp

template <int MODE>
__global__ void __launch_bounds__(kWarps * 32, 1) weights_kernel(KvWeightsArgs a, int lgG, int ways) {
  __shared__ float part[kWarps][kTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  const int j = (int)(blockIdx.y % a.Hkv);
  const int64_t b = blockIdx.y / a.Hkv;
  const int len = (int)min((int64_t)a.len[b], a.cap);
  const int R = (int)a.L << lgG;
  const int bi0 = (int)(b * a.L);
  const int tw = warp / ways, way = warp % ways;  // token group of the CTA, share of the rows
  const int t0 = (blockIdx.x * (kWarps / ways) + tw) * kTokens;
  const bool some = t0 < len;
  if ((int)(blockIdx.x * (kWarps / ways) * kTokens) >= len) return;  // the whole CTA

  float sum[4][2] = {};  // tokens 8 n + 2 tig, + 1
  if (some) {
    uint32_t kb[4][8][2];
    float f[4][2];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int t = t0 + 8 * n + gid;
      uint4 kh = make_uint4(0, 0, 0, 0), kl = kh;
      if (t < len) {
        const int64_t off = ((b * a.cap + t) * a.Hkv + j) * (kD / 2) + 16 * tig;
        kh = __ldg(reinterpret_cast<const uint4 *>(a.k_hi + off));
        if (MODE) kl = __ldg(reinterpret_cast<const uint4 *>(a.k_lo + off));
      }
      const uint32_t hw[4] = {kh.x, kh.y, kh.z, kh.w}, lw[4] = {kl.x, kl.y, kl.z, kl.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t ev, od;
        codes<MODE>(hw[w], lw[w], ev, od);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          kb[n][2 * w + h][0] = pair<MODE>(ev, od, 2 * h);
          kb[n][2 * w + h][1] = pair<MODE>(ev, od, 2 * h + 1);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = t0 + 8 * n + 2 * tig + i;
        f[n][i] = u < len ? half_bits(__ldg(a.k_scale + (b * a.cap + u) * a.Hkv + j)) *
                                (MODE ? 0.0625f * kScale : kScale)
                          : 0.0f;
      }
    }
    for (int r = way * 16; r < R; r += ways * 16) {
      const int r0 = r + gid, r1 = r0 + 8;
      const int64_t at0 = query_row(bi0, r0, lgG, (int)a.H, j), at1 = query_row(bi0, r1, lgG, (int)a.H, j);
      uint32_t qa[8][4];
      load_queries(qa, r0 < R ? a.q + at0 * kD : nullptr, r1 < R ? a.q + at1 * kD : nullptr, tig);
      // a row without weight (lse -inf) gives none
      const float e0 = r0 < R ? __ldg(a.lse + at0) : -INFINITY;
      const float e1 = r1 < R ? __ldg(a.lse + at1) : -INFINITY;
      const float b0 = e0 == -INFINITY ? INFINITY : e0 * kLog2e;
      const float b1 = e1 == -INFINITY ? INFINITY : e1 * kLog2e;
      // query i sees the tokens below len - L + 1 + i
      const int lim0 = len - (int)a.L + 1 + (r0 >> lgG);
      const int lim1 = len - (int)a.L + 1 + (r1 >> lgG);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_f16(d, qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], kb[n][ks][0], kb[n][ks][1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int u = t0 + 8 * n + 2 * tig + i;
          sum[n][i] += u < lim0 ? exp2_approx(fmaf(d[i], f[n][i], -b0)) : 0.0f;
          sum[n][i] += u < lim1 ? exp2_approx(fmaf(d[2 + i], f[n][i], -b1)) : 0.0f;
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v = sum[n][i];
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (gid == 0) part[warp][8 * n + 2 * tig + i] = v;
    }
  __syncthreads();
  const int span = (kWarps / ways) * kTokens;
  for (int e = threadIdx.x; e < span; e += kWarps * 32) {
    const int t = blockIdx.x * span + e;
    if (t >= len) continue;
    float v = 0.0f;
    for (int w = 0; w < ways; ++w) v += part[(e / kTokens) * ways + w][e % kTokens];
    a.acc[(b * a.Hkv + j) * a.cap + t] += v;
  }
}

// The same where a cache's rows are at most 128 (each sequence's own tokens
// mostly, and a shared prefix of a small batch): the rows' queries are held as A fragments in shared memory, and each warp brings
// 16 tokens at a time through a ring of asynchronous copies, so that the K
// planes stream in beside the products.  A CTA takes a part of one (cache,
// KV head)'s tokens; a token belongs to one warp, its sum to a fixed order.
constexpr int kOwnTile = 16, kStages = 3, kMostTiles = 8;
template <int MODE>
__global__ void __launch_bounds__(kWarps * 32, 3) few_rows_kernel(KvWeightsArgs a, int lgG, int splits,
                                                                     int part_len) {
  constexpr int kPlane = kOwnTile * (kD / 2), kStage = (MODE ? 2 : 1) * kPlane;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float base[kMostTiles * 16];  // -lse log2(e) of the rows, -inf for one without weight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const bool own = a.len != nullptr;  // else one cache, which every query sees whole
  const int Hkv = (int)a.Hkv, L = (int)(own ? a.L : a.B * a.L);
  const int R = L << lgG, row_tiles = (R + 15) / 16;
  const int bj = blockIdx.x / splits, split = blockIdx.x - bj * splits;
  const int b = bj / Hkv, j = bj - b * Hkv, bi0 = b * L;
  griddep_wait();
  griddep_launch_dependents();
  const int len = own ? min(a.len[b], (int)a.cap) : (int)a.cap;
  const int t_begin = split * part_len;
  if (t_begin >= len) return;
  const int t_end = min(len, t_begin + part_len);
  uint4 *frag = reinterpret_cast<uint4 *>(smem);
  const uint32_t ring = smem_u32(smem + row_tiles * kFrag + warp * kStages * kStage);

  // this lane's copies: pieces lane % 4 of rows lane / 4 and 8 + lane / 4; lane
  // l < 16 has token l's scale and sum so far
  const int64_t row_base = b * a.cap * Hkv + j;
  int t0 = t_begin + warp * kOwnTile;
  constexpr int kStep = kWarps * kOwnTile;
  const int64_t next = (int64_t)kStep * Hkv * (kD / 2), half = (int64_t)8 * Hkv * (kD / 2);
  int64_t off = (row_base + (int64_t)(t0 + gid) * Hkv) * (kD / 2) + 16 * tig;
  int t_load = t0;
  float *const acc = a.acc + (int64_t)bj * a.cap;
  auto load = [&](uint32_t at, uint16_t &scale, float &old) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const bool in = t_load + gid + 8 * n < t_end;
      const int64_t o = in ? off + n * half : 0;
      cp_async16(at + (gid + 8 * n) * (kD / 2) + 16 * tig, a.k_hi + o, in);
      if (MODE) cp_async16(at + kPlane + (gid + 8 * n) * (kD / 2) + 16 * tig, a.k_lo + o, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int t = t_load + (lane & 15);
    const bool in = t < t_end;
    scale = in ? __ldg(a.k_scale + row_base + (int64_t)t * Hkv) : (uint16_t)0;
    old = in ? acc[t] : 0.0f;
    off += next;
    t_load += kStep;
  };
  uint16_t sc[kStages];
  float old[kStages];
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i) load(ring + i * kStage, sc[i], old[i]);
  for (int r = warp; r < row_tiles; r += kWarps) {
    const int r0 = 16 * r + gid, r1 = r0 + 8;
    uint32_t qa[8][4];
    load_queries(qa, r0 < R ? a.q + query_row(bi0, r0, lgG, (int)a.H, j) * kD : nullptr,
                 r1 < R ? a.q + query_row(bi0, r1, lgG, (int)a.H, j) * kD : nullptr, tig);
    store_frag(frag + r * (kFrag / 16), qa, lane);
  }
  for (int r = threadIdx.x; r < 16 * row_tiles; r += kWarps * 32) {
    const float e = r < R ? a.lse[query_row(bi0, r, lgG, (int)a.H, j)] : -INFINITY;
    base[r] = e == -INFINITY ? -INFINITY : -e * kLog2e;
  }
  __syncthreads();

  for (int slot = 0; t0 < t_end; t0 += kStep) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();  // this tile is here, and every lane is done with the one before
    const int free = slot == 0 ? kStages - 1 : slot - 1;
    load(ring + free * kStage, sc[kStages - 1], old[kStages - 1]);
    const uint32_t cur = ring + slot * kStage;
    slot = slot == kStages - 1 ? 0 : slot + 1;
    float f[4], sum[4] = {};  // tokens 2 tig, 2 tig + 1, 8 + 2 tig, 9 + 2 tig
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 2 * tig + (i & 1) + 8 * (i >> 1);
      f[i] = half_bits((uint16_t)__shfl_sync(0xffffffffu, (int)sc[0], t)) * (MODE ? 0.0625f * kScale : kScale);
    }
    const float before = old[0];
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) {
      sc[i] = sc[i + 1];
      old[i] = old[i + 1];
    }
    uint4 u[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint4 h = lds128(cur + (8 * n + gid) * (kD / 2) + 16 * tig);
      const uint4 l = MODE ? lds128(cur + kPlane + (8 * n + gid) * (kD / 2) + 16 * tig) : make_uint4(0, 0, 0, 0);
      const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) u[n][w] = codes8<MODE>(hw[w], lw[w]);
    }
    const bool edge = own && t0 + kOwnTile > len - L + 1;  // some row does not see some token
    for (int r = 0; r < row_tiles; ++r) {
      float d[2][4] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4 q0 = frag[r * (kFrag / 16) + (2 * w) * 32 + lane],
                    q1 = frag[r * (kFrag / 16) + (2 * w + 1) * 32 + lane];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          mma_f16(d[n], q0.x, q0.y, q0.z, q0.w, u[n][w].x, u[n][w].y);
          mma_f16(d[n], q1.x, q1.y, q1.z, q1.w, u[n][w].z, u[n][w].w);
        }
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int row = 16 * r + 8 * g + gid;
        const float e = base[row];
        const int lim = edge ? len - L + 1 + (row >> lgG) : t_end;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 2 * tig + (i & 1) + 8 * (i >> 1);
          const float x = fmaf(d[i >> 1][2 * g + (i & 1)], f[i], e);
          if (t < lim) sum[i] += exp2_approx(x);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    // token l's sum to lane l
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = __shfl_sync(0xffffffffu, sum[i], (lane & 7) >> 1);
      if (i == (lane & 1) + 2 * ((lane >> 3) & 1)) v = s;
    }
    if (lane < 16 && t0 + lane < t_end) acc[t0 + lane] = before + v;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// --------------------------------------------------------------- eviction
constexpr int kSelect = 1024;

// Order of the accumulated weights as unsigned integers: greater weights have
// greater keys, -0 and 0 the same one, NaN the lowest.
__device__ __forceinline__ uint32_t key_of(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One CTA per (sequence, KV head): the kept tokens in increasing order.  The
// weight of the last one that is kept among those neither first nor recent is
// found from its key's bits, 8 at a time from the top (the count of each value
// of the next 8 bits among the tokens that share the bits so far); of the
// tokens with exactly that weight the first ones are kept.
//
// Weights crowd: many are 0, the others share a few exponents.  So each lane
// counts in a column of its own (32 KB: lanes of a warp never meet in a bank).
// Where at most 32 tokens are left to choose from, one warp's comparison ends
// the search, mostly after two rounds.
//
// A chunk is SPANS x 4096 tokens, four neighbours of each span for a thread:
// one scan over a chunk places its kept tokens.  A row of one chunk (HELD) is
// read once and stays in registers, a longer one is read again in each round.
template <int SPANS, bool HELD>
__global__ void __launch_bounds__(kSelect) select_kernel(KvEvictArgs a) {
  constexpr int kOwn = 4, kSpan = kSelect * kOwn, kChunk = SPANS * kSpan;
  static_assert(SPANS * kOwn <= 32 && kChunk < 65536, "masks of 32 bits, counts of 16");
  __shared__ __align__(16) int hist[256][32];
  __shared__ __align__(16) int total[256];
  __shared__ uint32_t sums[SPANS][32];  // by span and warp
  __shared__ uint32_t few[32];
  __shared__ int num_few, sh_want, sh_size;
  __shared__ uint32_t sh_prefix;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t bj = blockIdx.x, b = bj / a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = a.len[b];
  int32_t *kept = a.kept + bj * a.keep;
  if (bj % a.Hkv == 0 && tid == 0) a.len_out[b] = (int)min((int64_t)min((int64_t)len, a.cap), a.keep);
  if (len < 0) {  // the sequence is not taking part
    for (int64_t i = tid; i < a.keep; i += kSelect) kept[i] = -1;
    return;
  }
  const int n = (int)min((int64_t)len, a.cap);
  const float *acc = a.acc + bj * a.cap;
  float *acc_out = a.acc_out + bj * a.cap_out;
  const int keep = (int)min((int64_t)n, a.keep);
  const int first = (int)min(a.sinks, (int64_t)n), last = n - (int)min(a.recent, (int64_t)(n - first));
  int want = keep - first - (n - last);  // to choose among first .. last - 1
  const bool vec = (reinterpret_cast<uintptr_t>(acc) & 15) == 0;

  // keys of this thread's tokens of the chunk at `base`; bit 4 h + k of `mid`: token
  // base + h * kSpan + 4 tid + k is to be chosen from, of `in`: it is one of the n
  uint32_t key[SPANS][kOwn], mid, in;
  auto load = [&](int base) {
    mid = in = 0;
#pragma unroll
    for (int h = 0; h < SPANS; ++h) {
      const int i0 = base + h * kSpan + kOwn * tid;
      float v[kOwn];
      if (vec && i0 + kOwn <= n) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(acc + i0));
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
      } else {
#pragma unroll
        for (int k = 0; k < kOwn; ++k) v[k] = i0 + k < n ? __ldg(acc + i0 + k) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        key[h][k] = key_of(v[k]);
        in |= (uint32_t)(i0 + k < n) << (kOwn * h + k);
        mid |= (uint32_t)(i0 + k >= first && i0 + k < last) << (kOwn * h + k);
      }
    }
  };
  if (HELD) load(0);

  uint32_t prefix = 0;
  int equal = 0;  // how many with exactly the last kept weight
  if (n > a.keep && want > 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      reinterpret_cast<int4 *>(&hist[0][0])[tid + k * kSelect] = make_int4(0, 0, 0, 0);
    if (tid == 0) num_few = 0;
    __syncthreads();
    // f(key) for this thread's tokens to choose from whose key has the bits of
    // `prefix` that `mask` has
    uint32_t left = mid;  // HELD: those that had them in the last round
    auto each = [&](uint32_t mask, auto f) {
      for (int base = 0; base < (HELD ? 1 : last); base += kChunk) {
        if (!HELD) {
          load(base);
          left = mid;
        }
        if (left == 0) continue;
#pragma unroll
        for (int h = 0; h < SPANS; ++h)
#pragma unroll
          for (int k = 0; k < kOwn; ++k) {
            constexpr uint32_t one = 1;
            if (left & (one << (kOwn * h + k))) {
              if (((key[h][k] ^ prefix) & mask) == 0)
                f(key[h][k]);
              else
                left &= ~(one << (kOwn * h + k));
            }
          }
      }
    };
    for (int shift = 24; shift >= 0; shift -= 8) {
      each(shift == 24 ? 0u : 0xffffffffu << (shift + 8),
           [&](uint32_t k) { atomicAdd(&hist[(k >> shift) & 255u][lane], 1); });
      __syncthreads();
      if (tid < 256) {
        int sum = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // neighbours in different banks
          int4 *p = reinterpret_cast<int4 *>(hist[tid]) + ((tid + c) & 7);
          const int4 v = *p;
          sum += v.x + v.y + v.z + v.w;
          *p = make_int4(0, 0, 0, 0);
        }
        total[tid] = sum;
      }
      __syncthreads();
      if (warp == 0) {  // the value, from the greatest down: 8 of them a lane
        int t[8], mine = 0;
        const int4 lo4 = reinterpret_cast<const int4 *>(total)[62 - 2 * lane],
                   hi4 = reinterpret_cast<const int4 *>(total)[63 - 2 * lane];
        t[0] = hi4.w, t[1] = hi4.z, t[2] = hi4.y, t[3] = hi4.x;
        t[4] = lo4.w, t[5] = lo4.z, t[6] = lo4.y, t[7] = lo4.x;
#pragma unroll
        for (int q = 0; q < 8; ++q) mine += t[q];
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        int before = inc - mine;
        if (before < want && want <= inc) {  // one lane
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            if (before < want && want <= before + t[q]) {
              sh_prefix = prefix | ((uint32_t)(255 - (8 * lane + q)) << shift);
              sh_want = want - before;
              sh_size = t[q];
            }
            before += t[q];
          }
        }
      }
      __syncthreads();
      prefix = sh_prefix;
      want = sh_want;
      const int size = sh_size;
      if (shift > 0 && size <= 32) {
        each(0xffffffffu << shift, [&](uint32_t k) { few[atomicAdd(&num_few, 1)] = k; });
        __syncthreads();
        const uint32_t mine = lane < size ? few[lane] : 0u;
        int above = 0, same = 0;
        for (int i = 0; i < size; ++i) {
          const uint32_t o = __shfl_sync(0xffffffffu, mine, i);
          above += o > mine;
          same += o == mine;
        }
        const bool it = lane < size && above < want && want <= above + same;
        const int from = __ffs(__ballot_sync(0xffffffffu, it)) - 1;
        prefix = __shfl_sync(0xffffffffu, mine, from);
        want -= __shfl_sync(0xffffffffu, above, from);
        break;
      }
    }
    equal = want;
  }
  // the kept tokens, a chunk at a time: `done` taken so far for their weight or
  // place, `seen` with the last kept weight
  const bool all = n <= a.keep;
  int done = 0, seen = 0;
  for (int base = 0; base < n; base += kChunk) {
    if (!HELD) load(base);
    uint32_t take = all ? in : in & ~mid, tie = 0, inc[SPANS];
    if (equal > 0) {
#pragma unroll
      for (int h = 0; h < SPANS; ++h)
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
          take |= (uint32_t)(key[h][k] > prefix) << (kOwn * h + k) & mid;
          tie |= (uint32_t)(key[h][k] == prefix) << (kOwn * h + k) & mid;
        }
    }
    auto count = [&](int h) {  // ties << 16 | taken, of this thread in a span
      return (uint32_t)__popc(take >> (kOwn * h) & 15u) + ((uint32_t)__popc(tie >> (kOwn * h) & 15u) << 16);
    };
#pragma unroll
    for (int h = 0; h < SPANS; ++h) inc[h] = count(h);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int h = 0; h < SPANS; ++h) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, inc[h], o);
        if (lane >= o) inc[h] += x;
      }
    if (lane == 31)
#pragma unroll
      for (int h = 0; h < SPANS; ++h) sums[h][warp] = inc[h];
    __syncthreads();
    if (warp == 0) {  // exclusive sums over spans and warps
      uint32_t t[SPANS], before = 0;
#pragma unroll
      for (int h = 0; h < SPANS; ++h) {
        const uint32_t mine = sums[h][lane];
        t[h] = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, t[h], o);
          if (lane >= o) t[h] += x;
        }
        sums[h][lane] = before + t[h] - mine;
        before += __shfl_sync(0xffffffffu, t[h], 31);
      }
      if (lane == 0) total[0] = (int)before;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < SPANS; ++h) {
      const uint32_t ex = sums[h][warp] + inc[h] - count(h);
      int taken = done + (int)(ex & 0xffffu), ties = seen + (int)(ex >> 16);
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        const bool is_taken = take >> (kOwn * h + k) & 1u, is_tie = tie >> (kOwn * h + k) & 1u;
        if (is_taken || (is_tie && ties < equal)) {
          const int at = taken + min(ties, equal), i = base + h * kSpan + kOwn * tid + k;
          kept[at] = i;
          acc_out[at] = acc[i];  // its very bits, which the key may have lost
        }
        taken += is_taken;
        ties += is_tie;
      }
    }
    done += total[0] & 0xffff;
    seen += (int)((uint32_t)total[0] >> 16);
    __syncthreads();  // sums and total may be written again
  }
  for (int64_t i = keep + tid; i < a.keep; i += kSelect) kept[i] = -1;
  for (int64_t i = keep + tid; i < a.cap_out; i += kSelect) acc_out[i] = 0.0f;
}

// Rows of the kept tokens into the new cache: 16 lanes take kRun kept tokens of
// one KV head, 16 bytes of one of the four planes a lane; the first two carry
// the scales.  The kRun loads of a lane are in flight together.
constexpr int kRun = 8;
// Rows of one head lie 64 bytes in every Hkv * 64: by default DRAM is read in
// pieces of 128 (16 x 8 x 32768 tokens cut to a quarter: 449 MB and 107 us, 287
// MB and 103 us with this).
__device__ __forceinline__ uint4 load_64(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::64B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__global__ void __launch_bounds__(256) gather_kernel(KvEvictArgs a, int runs) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int l = (int)(id & 15);
  const int64_t r = id >> 4;  // (b * runs + run) * Hkv + j: neighbours write neighbouring rows
  if (r >= a.B * runs * a.Hkv) return;
  const int64_t j = r % a.Hkv, br = r / a.Hkv, run = br % runs, b = br / runs;
  const int32_t *kept = a.kept + (b * a.Hkv + j) * a.keep + run * kRun;
  const int left = (int)min((int64_t)kRun, a.keep - run * kRun);
  const int plane = l >> 2, piece = l & 3;
  const uint8_t *s = plane == 0 ? a.src.k_hi : plane == 1 ? a.src.k_lo : plane == 2 ? a.src.v_hi : a.src.v_lo;
  uint8_t *d = plane == 0 ? a.dst.k_hi : plane == 1 ? a.dst.k_lo : plane == 2 ? a.dst.v_hi : a.dst.v_lo;
  const uint16_t *ss = l == 0 ? a.src.k_scale : a.src.v_scale;
  uint16_t *ds = l == 0 ? a.dst.k_scale : a.dst.v_scale;
  int t[kRun];
  uint4 w[kRun];
  uint16_t sc[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) t[i] = i < left ? kept[i] : -1;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int64_t from = (b * a.cap + max(t[i], 0)) * a.Hkv + j;
    if (t[i] >= 0) {
      w[i] = load_64(reinterpret_cast<const uint4 *>(s + from * (kD / 2)) + piece);
      if (l < 2) sc[i] = __ldg(ss + from);
    }
  }
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int64_t to = (b * a.cap_out + run * kRun + i) * a.Hkv + j;
    if (t[i] >= 0) {
      reinterpret_cast<uint4 *>(d + to * (kD / 2))[piece] = w[i];
      if (l < 2) ds[to] = sc[i];
    }
  }
}

}  // namespace evict

// From this many rows on a shared cache is on the tensor cores' tcgen05 path:
// with 8 KV heads and 16384 tokens that takes 17.9 us at any number of rows up to
// 128, few_rows_kernel 17.7 at 96 and 21.9 at 128; with one KV head and 512 tokens
// 5.2 against 4.4 and 5.2.
constexpr int64_t kTcRows = 128;

cudaError_t launch_kv_weights(const KvWeightsArgs &a, cudaStream_t st) {
  const int G = (int)(a.H / a.Hkv);
  const int64_t R = (a.len ? a.L : a.B * a.L) * G;
  if (!a.len && R >= kTcRows) return evict::launch_weights_tc(a, st);
  int lgG = 0;
  while ((1 << lgG) < G) ++lgG;
  const int64_t caches = (a.len ? a.B : 1) * a.Hkv;
  if (R <= 16 * evict::kMostTiles) {
    // One CTA an SM with few tokens each, nine with more: two tiles a warp, three CTAs
    // an SM at a time.  Lengths differ, so many small parts share the SMs better: 16 x 8
    // caches of 0 to 4096 tokens take 15.7 us, 17.4 with four tiles a warp and three
    // CTAs an SM, 21.9 with two.
    const int64_t step = evict::kWarps * evict::kOwnTile;
    int64_t s = std::max((148 + caches - 1) / caches, std::min((9 * 148 + caches - 1) / caches, a.cap / (2 * step)));
    s = std::max((int64_t)1, std::min(s, (a.cap + step - 1) / step));
    const int64_t part = ((a.cap + s - 1) / s + step - 1) / step * step;
    const int splits = (int)((a.cap + part - 1) / part), tiles = (int)((R + 15) / 16);
    auto kern = a.mode ? evict::few_rows_kernel<1> : evict::few_rows_kernel<0>;
    const int ring = evict::kWarps * evict::kStages * (a.mode ? 2 : 1) * evict::kOwnTile * 64;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         evict::kMostTiles * nested::kFrag + ring);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)(caches * splits)), dim3(evict::kWarps * 32),
                      tiles * nested::kFrag + ring, st, true, a, lgG, splits, (int)part);
  }
  // The warps of a CTA share the rows of its tokens when there are more rows
  // than a warp's pass and too few tokens to give every warp its own.
  int ways = 1;
  while (ways < evict::kWarps && R > 16 * ways &&
         caches * ((a.cap + evict::kTokens - 1) / evict::kTokens) < 2 * 148 * (evict::kWarps / ways))
    ways *= 2;
  const int64_t span = (evict::kWarps / ways) * evict::kTokens;
  const dim3 grid((unsigned)((a.cap + span - 1) / span), (unsigned)caches);
  auto kern = a.mode ? evict::weights_kernel<1> : evict::weights_kernel<0>;
  return launch_pdl(kern, grid, dim3(evict::kWarps * 32), 0, st, true, a, lgG, ways);
}

cudaError_t launch_kv_evict(const KvEvictArgs &a, cudaStream_t st) {
  auto select = a.cap <= 4096    ? evict::select_kernel<1, true>
                : a.cap <= 8192  ? evict::select_kernel<2, true>
                : a.cap <= 32768 ? evict::select_kernel<8, true>
                                 : evict::select_kernel<8, false>;
  cudaError_t e = launch_pdl(select, dim3((unsigned)(a.B * a.Hkv)), dim3(evict::kSelect), 0, st, true, a);
  if (e != cudaSuccess) return e;
  const int64_t runs = (a.keep + evict::kRun - 1) / evict::kRun;
  const int64_t blocks = (a.B * runs * a.Hkv * 16 + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(evict::gather_kernel, dim3((unsigned)blocks), dim3(256), 0, st, true, a, (int)runs);
}

}  // namespace bitnest
