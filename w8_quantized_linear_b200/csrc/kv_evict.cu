// A bounded nested KV cache: the attention weight each cached token has
// received, and eviction of the tokens that received least.
#include "launch.h"
#include "nested_mma.cuh"

namespace bitnest {

namespace evict {

using namespace nested;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kScale = 0.088388347648318440550f * kLog2e;  // log2(e) / sqrt(128)

// ---------------------------------------------------------------- weights
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
  const bool own = a.len != nullptr;
  const int j = (int)(blockIdx.y % a.Hkv);
  const int64_t b = blockIdx.y / a.Hkv;  // 0 where the cache is shared
  const int len = own ? (int)min((int64_t)a.len[b], a.cap) : (int)a.cap;
  const int R = (int)(own ? a.L : a.B * a.L) << lgG;
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
      // own tokens: query i sees those below len - L + 1 + i
      const int lim0 = own ? len - (int)a.L + 1 + (r0 >> lgG) : len;
      const int lim1 = own ? len - (int)a.L + 1 + (r1 >> lgG) : len;
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
      w[i] = __ldg(reinterpret_cast<const uint4 *>(s + from * (kD / 2)) + piece);
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

cudaError_t launch_kv_weights(const KvWeightsArgs &a, cudaStream_t st) {
  const int G = (int)(a.H / a.Hkv);
  const int64_t R = (a.len ? a.L : a.B * a.L) * G;
  if (!a.len && R >= 128 && a.Hkv * ((a.cap + 127) / 128) <= 0x3fffffff)
    return evict::launch_weights_tc(a, st);
  int lgG = 0;
  while ((1 << lgG) < G) ++lgG;
  // The warps of a CTA share the rows of its tokens when there are more rows
  // than a warp's pass and too few tokens to give every warp its own.
  const int64_t caches = (a.len ? a.B : 1) * a.Hkv;
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
