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
__global__ void __launch_bounds__(kWarps * 32, 1) weights_kernel(KvWeightsArgs a, int G, int ways) {
  __shared__ float part[kWarps][kTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  const bool own = a.len != nullptr;
  const int j = (int)(blockIdx.y % a.Hkv);
  const int64_t b = blockIdx.y / a.Hkv;  // 0 where the cache is shared
  const int len = own ? (int)min((int64_t)a.len[b], a.cap) : (int)a.cap;
  const int R = (int)((own ? a.L : a.B * a.L) * G);
  const int64_t bi0 = b * a.L;
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
      const int64_t at0 = query_row(bi0, r0, G, a.H, j), at1 = query_row(bi0, r1, G, a.H, j);
      uint32_t qa[8][4];
      load_queries(qa, r0 < R ? a.q + at0 * kD : nullptr, r1 < R ? a.q + at1 * kD : nullptr, tig);
      // a row without weight (lse -inf) gives none
      const float e0 = r0 < R ? __ldg(a.lse + at0) : -INFINITY;
      const float e1 = r1 < R ? __ldg(a.lse + at1) : -INFINITY;
      const float b0 = e0 == -INFINITY ? INFINITY : e0 * kLog2e;
      const float b1 = e1 == -INFINITY ? INFINITY : e1 * kLog2e;
      // own tokens: query i sees those below len - L + 1 + i
      const int lim0 = own ? len - (int)a.L + 1 + r0 / G : len;
      const int lim1 = own ? len - (int)a.L + 1 + r1 / G : len;
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

// Sum of v over the block, and the sum over the threads before this one.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int s = warp_sums[lane];  // 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += x;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  __syncthreads();  // warp_sums may be written again
  return inc - v + (warp > 0 ? before : 0);
}

// One CTA per (sequence, KV head): the kept tokens in increasing order.  The
// weight of the last one that is kept among those neither first nor recent is
// found from its key's bits, 8 at a time from the top (the count of each value
// of the next 8 bits among the tokens that share the bits so far); of the
// tokens with exactly that weight the first ones are kept.
__global__ void __launch_bounds__(kSelect) select_kernel(KvEvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_want;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t bj = blockIdx.x, b = bj / a.Hkv;
  const int tid = threadIdx.x;
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
  uint32_t prefix = 0;
  int equal = 0;  // how many with exactly the last kept weight
  if (n > a.keep && want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = first + tid; i < last; i += kSelect) {
        const uint32_t k = key_of(acc[i]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(k >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid < 32) {  // from the greatest value down: 8 values a lane
        int mine = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) mine += hist[255 - (8 * tid + q)];
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, inc, o);
          if (tid >= o) inc += x;
        }
        int before = inc - mine;
        if (before < want && want <= inc) {
          for (int q = 0; q < 8; ++q) {
            const int v = 255 - (8 * tid + q);
            if (before + hist[v] >= want) {
              sh_prefix = prefix | ((uint32_t)v << shift);
              sh_want = want - before;
              break;
            }
            before += hist[v];
          }
        }
      }
      __syncthreads();
      prefix = sh_prefix;
      want = sh_want;
    }
    equal = want;
  }
  // the kept tokens, 1024 at a time, in order
  int done = 0, seen = 0;  // kept so far, and with the last kept weight so far
  for (int base = 0; base < n; base += kSelect) {
    const int i = base + tid;
    int take = 0, tie = 0;
    float v = 0.0f;
    if (i < n) {
      v = acc[i];
      if (n <= a.keep || i < first || i >= last) {
        take = 1;
      } else if (equal > 0) {
        const uint32_t k = key_of(v);
        take = k > prefix;
        tie = k == prefix;
      }
    }
    int ties, total;
    const int tie_rank = seen + block_scan(tie, warp_sums, &ties);
    if (tie && tie_rank < equal) take = 1;
    const int at = done + block_scan(take, warp_sums, &total);
    if (take) {
      kept[at] = i;
      acc_out[at] = v;
    }
    seen += ties;
    done += total;
  }
  for (int64_t i = done + tid; i < a.keep; i += kSelect) kept[i] = -1;
  for (int64_t i = done + tid; i < a.cap_out; i += kSelect) acc_out[i] = 0.0f;
}

// Rows of the kept tokens into the new cache: 16 lanes a row, 16 bytes of one
// of the four planes each; the first two carry the scales.
__global__ void __launch_bounds__(256) gather_kernel(KvEvictArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int l = (int)(id & 15);
  const int64_t r = id >> 4;  // (b * keep + at) * Hkv + j
  if (r >= a.B * a.keep * a.Hkv) return;
  const int64_t j = r % a.Hkv, bt = r / a.Hkv, at = bt % a.keep, b = bt / a.keep;
  const int t = a.kept[(b * a.Hkv + j) * a.keep + at];
  if (t < 0) return;
  const int64_t from = (b * a.cap + t) * a.Hkv + j, to = (b * a.cap_out + at) * a.Hkv + j;
  const int plane = l >> 2, piece = l & 3;
  const uint8_t *s = plane == 0 ? a.src.k_hi : plane == 1 ? a.src.k_lo : plane == 2 ? a.src.v_hi : a.src.v_lo;
  uint8_t *d = plane == 0 ? a.dst.k_hi : plane == 1 ? a.dst.k_lo : plane == 2 ? a.dst.v_hi : a.dst.v_lo;
  reinterpret_cast<uint4 *>(d + to * (kD / 2))[piece] =
      __ldg(reinterpret_cast<const uint4 *>(s + from * (kD / 2)) + piece);
  if (l == 0) a.dst.k_scale[to] = a.src.k_scale[from];
  if (l == 1) a.dst.v_scale[to] = a.src.v_scale[from];
}

}  // namespace evict

cudaError_t launch_kv_weights(const KvWeightsArgs &a, cudaStream_t st) {
  const int G = (int)(a.H / a.Hkv);
  const int64_t R = (a.len ? a.L : a.B * a.L) * G;
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
  return launch_pdl(kern, grid, dim3(evict::kWarps * 32), 0, st, true, a, G, ways);
}

cudaError_t launch_kv_evict(const KvEvictArgs &a, cudaStream_t st) {
  cudaError_t e = launch_pdl(evict::select_kernel, dim3((unsigned)(a.B * a.Hkv)),
                             dim3(evict::kSelect), 0, st, true, a);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.B * a.keep * a.Hkv * 16 + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(evict::gather_kernel, dim3((unsigned)blocks), dim3(256), 0, st, true, a);
}

}  // namespace bitnest
