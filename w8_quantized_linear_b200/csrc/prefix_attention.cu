// Attention of a batch of sequences that share a prefix, over nested KV
// caches: query i of sequence b (of L) attends over the P prefix tokens, which
// are stored once, and over its own cached tokens t <= len[b] - L + i,
//   o = sum_t p_t v_t,  p = softmax(q k_t / sqrt(128)).
//
// The softmax is split by tokens: each part of the tokens gives its own
// maximum, sum and output, and parts join by
//   m = max m_s,  l = sum l_s 2^(m_s - m),  o = sum o_s l_s 2^(m_s - m) / l.
// So the prefix is attended by all rows (queries x heads of a KV head) of the
// batch together, as one product per KV head, and each sequence's own tokens
// by its rows only; a second kernel joins the parts.
//
// Bound of the parts on mma.sync: instructions (counted for a warp's 16 target
// tokens: 662 with 16 rows, 523 with 8; 572 and 450 for draft tokens; a good part of
// them unpacks codes) and, in small calls, latency: 2 queries over 2048 + 128 draft
// tokens take 7.1 us with the join, 16 x 8 caches of 0 to 1024 target tokens 19 us
// with it (17 MB, 2.6 us to read).
#include "launch.h"
#include "nested_mma.cuh"
#include "prefix_plan.h"
#include "sm100.cuh"

namespace bitnest {

namespace pattn {

using namespace nested;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;   // tokens a warp takes at a time
constexpr int kRows = 16;   // rows of a warp
constexpr int kMinExp = -40;  // below any fp16 scale / 16
constexpr float kSlack = 8.0f;
constexpr int kHead = 7;  // p v_scale < 2^(8 + 7)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kScale = 0.088388347648318440550f * kLog2e;  // log2(e) / sqrt(128)

// Shared memory of a CTA: the rows' queries as A fragments (4 KB a row tile),
// then each warp's ring of token tiles; the ring's place holds the warps'
// states when they join.
constexpr int kStages = 3;
__host__ __device__ constexpr int stage_bytes(int mode) { return (mode ? 4 : 2) * kTile * (kD / 2); }
struct State {
  float m[kWarps][kRows], l[kWarps][kRows];
  float4 o[kWarps][8][2][32];  // as a lane holds it: [columns tile][rows tile][lane]
};
constexpr int smem_bytes(int mode, int row_tiles) {
  const int ring = kWarps * kStages * stage_bytes(mode);
  return row_tiles * kFrag + (ring > (int)sizeof(State) ? ring : (int)sizeof(State));
}

// A warp's way through a cache's rows, for one lane: of each plane's tile it
// copies the 16-byte pieces lane % 4 of rows lane / 4 and 8 + lane / 4, and it
// reads the scale of K (lanes 0 to 15) or V (16 to 31) of token lane % 16.  A
// row's pieces lie together; V's are exchanged so that the lanes that read a
// column's 8 bytes of four row pairs find them in different banks.  Tokens at
// or past the end are zeros.
template <int MODE>
struct Loader {
  static constexpr int kPlane = kTile * (kD / 2);
  const KvPlanes &c;
  const uint16_t *scale;
  int64_t off, next, half, scale_off, scale_next;  // bytes, and scales
  int t, end, stride;                              // row lane / 4's token
  uint32_t kd, vd[2];
  __device__ __forceinline__ Loader(const KvPlanes &c, int t0, int t_end, int step_tokens,
                                    int64_t row_base, int Hkv, int lane)
      : c(c), end(t_end), stride(step_tokens) {
    const int r = lane >> 2, p = lane & 3;
    t = t0 + r;
    off = (row_base + (int64_t)t * Hkv) * (kD / 2) + 16 * p;
    next = (int64_t)step_tokens * Hkv * (kD / 2);
    half = (int64_t)8 * Hkv * (kD / 2);
    scale = lane < 16 ? c.k_scale : c.v_scale;
    scale_off = row_base + (int64_t)(t0 + (lane & 15)) * Hkv;
    scale_next = (int64_t)step_tokens * Hkv;
    kd = r * (kD / 2) + 16 * p;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int q = r + 8 * n;
      vd[n] = (MODE ? 2 : 1) * kPlane + (q >> 1) * kD +
              16 * ((((q & 1) << 2) | p) ^ (((q >> 1) & 3) << 1));
    }
  }
  // The next tile into the stage at `at`; its scale.
  __device__ __forceinline__ uint16_t operator()(uint32_t at, int lane) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const bool in = t + 8 * n < end;
      const int64_t o = in ? off + n * half : 0;
      cp_async16(at + kd + n * 8 * (kD / 2), c.k_hi + o, in);
      if (MODE) cp_async16(at + kd + n * 8 * (kD / 2) + kPlane, c.k_lo + o, in);
      cp_async16(at + vd[n], c.v_hi + o, in);
      if (MODE) cp_async16(at + vd[n] + kPlane, c.v_lo + o, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    uint16_t s = 0;
    if (t - (lane >> 2) + (lane & 15) < end) s = __ldg(scale + scale_off);
    t += stride;
    off += next;
    scale_off += scale_next;
    return s;
  }
};

// One part for a tile of 16 rows (queries at `frag`): every tile of `load`, row
// r seeing tokens below lim(r).  As on the tcgen05 path p is kept as 2^(s -
// shift), shift = m + e - kHead with m a maximum at most kSlack behind and 2^e
// above every V scale so far: the output is rescaled only when one of them has
// grown, and p v_scale < 2^15 enters the product as two fp16 terms (22 bits
// together; one alone would put 2^-11 of every weight into outputs that cancel).
// e with vmax < 2^e, at most 100 (an infinite scale)
__device__ __forceinline__ int e_tile_of(float vmax) {
  return vmax > 0.0f ? min(100, (int)((__float_as_uint(vmax) >> 23) & 0xFFu) - 126) : kMinExp;
}
template <int NT>  // row tiles of 8: 1 where there are no more than 8 rows
struct Part {
  float shift[NT], l_run[NT];  // rows lane / 4, + 8
  float o[8][NT][4];           // O^T: columns tile mt, rows tile nt
};
template <int MODE, int NT>
__device__ __forceinline__ void attend(Part<NT> &st, const uint4 *frag, Loader<MODE> &load,
                                       uint32_t ring, uint16_t (&sc)[kStages], int lane, int t0,
                                       int t_end, int stride, const int (&seen_to)[2]) {
  constexpr int kPlane = kTile * (kD / 2);
  const int gid = lane >> 2, tig = lane & 3;
  float(&shift)[NT] = st.shift, (&l_run)[NT] = st.l_run, (&o)[8][NT][4] = st.o;
  float m[NT];
  int lim[NT], e_run = kMinExp;
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    lim[r] = min(seen_to[r], t_end);
    m[r] = -INFINITY;
    shift[r] = l_run[r] = 0.0f;
  }
#pragma unroll
  for (int mt = 0; mt < 8; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.0f;

  for (int slot = 0; t0 < t_end; t0 += stride) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();  // this tile is here, and every lane is done with the one before
    const int free = slot == 0 ? kStages - 1 : slot - 1;
    sc[kStages - 1] = load(ring + free * stage_bytes(MODE), lane);
    const uint32_t cur = ring + slot * stage_bytes(MODE);
    slot = slot == kStages - 1 ? 0 : slot + 1;
    uint16_t ks[4], vs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 2 * tig + (i & 1) + 8 * (i >> 1);
      ks[i] = (uint16_t)__shfl_sync(0xffffffffu, (int)sc[0], t);
      vs[i] = (uint16_t)__shfl_sync(0xffffffffu, (int)sc[0], 16 + t);
    }
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) sc[i] = sc[i + 1];
    float s[NT][4];  // [row][token 2 tig, 2 tig + 1, 8 + 2 tig, 9 + 2 tig]
    {
      uint4 kh[2], kl[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        kh[n] = lds128(cur + (8 * n + gid) * (kD / 2) + 16 * tig);
        kl[n] = MODE ? lds128(cur + kPlane + (8 * n + gid) * (kD / 2) + 16 * tig) : make_uint4(0, 0, 0, 0);
      }
      float d[2][4] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4 q0 = frag[(2 * w) * 32 + lane], q1 = frag[(2 * w + 1) * 32 + lane];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t hw[4] = {kh[n].x, kh[n].y, kh[n].z, kh[n].w};
          const uint32_t lw[4] = {kl[n].x, kl[n].y, kl[n].z, kl[n].w};
          const uint4 u = codes8<MODE>(hw[w], lw[w]);
          mma_f16(d[n], q0.x, q0.y, q0.z, q0.w, u.x, u.y);
          mma_f16(d[n], q1.x, q1.y, q1.z, q1.w, u.z, u.w);
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int r = 0; r < NT; ++r) {
          s[r][2 * n] = d[n][2 * r];
          s[r][2 * n + 1] = d[n][2 * r + 1];
        }
      }
    }
    float vf[4], vmax = 0.0f, tmax[NT];
#pragma unroll
    for (int r = 0; r < NT; ++r) tmax[r] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 2 * tig + (i & 1) + 8 * (i >> 1);
      const float f = half_bits(ks[i]) * (MODE ? 0.0625f * kScale : kScale);
      vf[i] = half_bits(vs[i]) * (MODE ? 0.0625f : 1.0f);
      vmax = fmaxf(vmax, vf[i]);
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        // a token that a row does not see counts as -inf whatever its scale holds
        s[r][i] = t < lim[r] ? s[r][i] * f : -INFINITY;
        tmax[r] = fmaxf(tmax[r], s[r][i]);
      }
    }
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) {
      vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, x));
#pragma unroll
      for (int r = 0; r < NT; ++r) tmax[r] = fmaxf(tmax[r], __shfl_xor_sync(0xffffffffu, tmax[r], x));
    }
    bool grown = e_tile_of(vmax) > e_run;
#pragma unroll
    for (int r = 0; r < NT; ++r) grown |= tmax[r] > m[r] + kSlack;
    if (__any_sync(0xffffffffu, grown)) {
      const int e_new = max(e_run, e_tile_of(vmax));
      float corr[NT];
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        const float old = shift[r];
        const bool fresh = m[r] == -INFINITY;  // a row that has seen no token: nothing to rescale
        if (tmax[r] > m[r] + kSlack) m[r] = tmax[r];
        shift[r] = m[r] == -INFINITY ? 0.0f : m[r] + (float)(e_new - kHead);
        corr[r] = fresh ? 1.0f : exp2_approx(old - shift[r]);
        l_run[r] *= corr[r];
      }
      e_run = e_new;
      // rows 8 nt + 2 tig, + 1 of O^T's columns: their corr is in lanes 8 tig, 8 tig + 4
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float c0 = __shfl_sync(0xffffffffu, corr[nt], 8 * tig);
        const float c1 = __shfl_sync(0xffffffffu, corr[nt], 8 * tig + 4);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          o[mt][nt][0] *= c0;
          o[mt][nt][1] *= c1;
          o[mt][nt][2] *= c0;
          o[mt][nt][3] *= c1;
        }
      }
    }
    uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      float p[4], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool seen = s[r][i] != -INFINITY;
        p[i] = seen ? exp2_approx(s[r][i] - shift[r]) : 0.0f;
        sum += p[i];
        p[i] = seen ? p[i] * vf[i] : 0.0f;
      }
      l_run[r] += sum;  // this lane's tokens only
      pb[r][0] = split_half2(p[0], p[1], pl[r][0]);
      pb[r][1] = split_half2(p[2], p[3], pl[r][1]);
    }
    uint32_t ev[4][2], od[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 2 * tig + (i & 1) + 8 * (i >> 1);  // 8 bytes at 8 gid of this token's row
      const uint32_t at = cur + (MODE ? 2 : 1) * kPlane + (r >> 1) * kD + 8 * (gid & 1) +
                          16 * ((((r & 1) << 2) | (gid >> 1)) ^ (((r >> 1) & 3) << 1));
      const uint2 vh = lds64(at), vl = MODE ? lds64(at + kPlane) : make_uint2(0, 0);
      codes<MODE>(vh.x, vl.x, ev[i][0], od[i][0]);
      codes<MODE>(vh.y, vl.y, ev[i][1], od[i][1]);
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // plane bytes 8 gid + 2 h, + 1: columns 16 gid + 4 h .. + 3
      const int w = h >> 1, b = 2 * (h & 1);
      uint32_t a[4][2];
      pair2<MODE>(a[0], ev[0][w], ev[1][w], b);
      pair2<MODE>(a[1], od[0][w], od[1][w], b);
      pair2<MODE>(a[2], ev[2][w], ev[3][w], b);
      pair2<MODE>(a[3], od[2][w], od[3][w], b);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(o[2 * h + i][nt], a[0][i], a[1][i], a[2][i], a[3][i], pb[nt][0], pb[nt][1]);
          mma_f16(o[2 * h + i][nt], a[0][i], a[1][i], a[2][i], a[3][i], pl[nt][0], pl[nt][1]);
        }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The state into slot `warp` of the shared memory.
template <int NT>
__device__ __forceinline__ void store_state(State &sh, Part<NT> &st, int warp, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    st.l_run[r] += __shfl_xor_sync(0xffffffffu, st.l_run[r], 1);
    st.l_run[r] += __shfl_xor_sync(0xffffffffu, st.l_run[r], 2);
    if (tig == 0) {
      sh.m[warp][gid + 8 * r] = st.shift[r];
      sh.l[warp][gid + 8 * r] = st.l_run[r];
    }
  }
#pragma unroll
  for (int mt = 0; mt < 8; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      sh.o[warp][mt][nt][lane] = make_float4(st.o[mt][nt][0], st.o[mt][nt][1], st.o[mt][nt][2], st.o[mt][nt][3]);
}

// The parts: CTAs below p_ctas take (KV head, row group, part of the prefix),
// the others (sequence, KV head, row tile, part of its own tokens).
// part_lse [parts, B L H] (in units of log 2), part_o [parts, B L H, 128].
template <int MODE, int NT>
__global__ void __launch_bounds__(kThreads, 2) parts_kernel(PrefixAttnArgs a, Plan pl,
                                                            float *__restrict__ part_lse,
                                                            float *__restrict__ part_o) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2;
  const int H = (int)a.H, L = (int)a.L, Hkv = (int)a.Hkv, lgG = pl.lgG;
  const int64_t rows_out = a.B * a.L * H;
  // Behind the tcgen05 kernel this one does not wait for it: that one began
  // (and let this one begin) when all before it was complete.  Ending after it,
  // as the join needs, is enough.
  if (!pl.tc) griddep_wait();
  griddep_launch_dependents();
  int cta = blockIdx.x;
  const bool prefix = cta < pl.p_ctas;
  int j, row0, R, t_begin, t_end, ways, row_warps, part, bi0;
  int64_t row_base;
  int visible;  // own: tokens that the sequence's query 0 sees
  if (prefix) {
    int rest = cta / pl.p_splits;
    const int split = cta - rest * pl.p_splits;
    j = rest / pl.p_groups;
    row_warps = pl.row_warps;
    row0 = (rest - j * pl.p_groups) * row_warps * kRows;
    R = (int)a.B * L << lgG;
    bi0 = 0;
    row_base = j;
    t_begin = split * pl.p_len;
    t_end = min((int)a.P, t_begin + pl.p_len);
    part = split;
    visible = (int)a.P;
  } else {
    cta -= pl.p_ctas;
    int rest = cta / pl.o_splits;
    const int split = cta - rest * pl.o_splits;
    int bj = rest / pl.o_tiles;
    row0 = (rest - bj * pl.o_tiles) * kRows;
    const int b = bj / Hkv;
    j = bj - b * Hkv;
    row_warps = 1;
    R = L << lgG;
    bi0 = b * L;
    row_base = b * a.cap * Hkv + j;
    const int len = min(__ldg(a.len + b), (int)a.cap);
    t_begin = split * pl.o_len;
    if (t_begin >= len) {  // no tokens: no weight (nothing reads the parts of len < 0)
      const int r = row0 + (int)threadIdx.x;
      if (threadIdx.x < kRows && r < R)
        part_lse[(int64_t)(pl.p_splits + split) * rows_out + query_row(bi0, r, lgG, H, j)] = -INFINITY;
      if (pl.tc) griddep_wait();
      return;
    }
    t_end = min(len, t_begin + pl.o_len);
    part = pl.p_splits + split;
    visible = len - L + 1;
  }
  ways = kWarps / row_warps;
  const int rw = warp % row_warps, way = warp / row_warps;
  const int r0 = row0 + rw * kRows + gid, r1 = r0 + 8;
  const int seen_to[2] = {r0 >= R ? 0 : prefix ? visible : visible + (r0 >> lgG),
                          r1 >= R ? 0 : prefix ? visible : visible + (r1 >> lgG)};
  uint4 *frag = reinterpret_cast<uint4 *>(smem_raw + rw * kFrag);
  uint8_t *rest = smem_raw + row_warps * kFrag;
  const uint32_t ring = smem_u32(rest + warp * kStages * stage_bytes(MODE));
  uint32_t qa[8][4];  // first, not behind the ring's burst
  if (way == 0)
    load_queries(qa, r0 < R ? a.q + query_row(bi0, r0, lgG, H, j) * kD : nullptr,
                 r1 < R ? a.q + query_row(bi0, r1, lgG, H, j) * kD : nullptr, lane & 3);
  const int t0 = t_begin + way * kTile, stride = ways * kTile;
  Loader<MODE> load(prefix ? a.prefix : a.own, t0, t_end, stride, row_base, Hkv, lane);
  uint16_t sc[kStages];  // scales of the tiles in the ring, the oldest first
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i) sc[i] = load(ring + i * stage_bytes(MODE), lane);
  if (way == 0) {
    store_frag(frag, qa, lane);
  }
  __syncthreads();
  Part<NT> st;
  attend<MODE, NT>(st, frag, load, ring, sc, lane, t0, t_end, stride, seen_to);
  __syncthreads();  // the ring's place is free
  State &sh = *reinterpret_cast<State *>(rest);
  store_state(sh, st, warp, lane);
  __syncthreads();
  // the warps' states joined by rows' factors 2^(shift_w - M) / den (0 for a
  // warp that saw no token; NaN scores make l NaN): 128 rows x ways, a thread each of
  // the first four warps
  if (warp < 4) {
    const int t = threadIdx.x, k = t & (ways - 1), row = t / ways;
    const int w = row / kRows + k * row_warps, rr = row % kRows, r = row0 + row;
    const bool in = rr < 8 * NT;
    const float l = in ? sh.l[w][rr] : 0.0f, m = in ? sh.m[w][rr] : 0.0f;
    float M = l != 0.0f ? m : -INFINITY;
    for (int x = 1; x < ways; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    const float f = l == 0.0f ? 0.0f : exp2_approx(m - M);
    float den = f * l;
    for (int x = 1; x < ways; x <<= 1) den += __shfl_xor_sync(0xffffffffu, den, x);
    __syncwarp();
    if (in) {
      sh.m[w][rr] = den == 0.0f ? 0.0f : f / den;
      if (k == 0 && r < R)
        part_lse[(int64_t)part * rows_out + query_row(bi0, r, lgG, H, j)] =
            den == 0.0f ? -INFINITY : M + log2f(den);
    }
  }
  __syncthreads();
  // a thread has two rows (8 nt + 2 (lane % 4), + 1) and four columns (16 (lane / 4)
  // + 4 mp ..) of a row tile at a time
  for (int e = threadIdx.x; e < row_warps * NT * 4 * 32; e += kThreads) {
    const int l = e & 31, mp = (e >> 5) & 3, nt = (e >> 7) & (NT - 1), w0 = e / (NT * 128);
    const int rr = 8 * nt + 2 * (l & 3), r0 = row0 + w0 * kRows + rr;
    if (r0 >= R) continue;
    float num[2][4] = {};
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const int w = w0 + k * row_warps;
      if (w >= kWarps) break;
      const float4 a4 = sh.o[w][2 * mp][nt][l], b4 = sh.o[w][2 * mp + 1][nt][l];
      const float2 f = *reinterpret_cast<const float2 *>(&sh.m[w][rr]);
      num[0][0] += f.x * a4.x;
      num[0][1] += f.x * a4.z;
      num[0][2] += f.x * b4.x;
      num[0][3] += f.x * b4.z;
      num[1][0] += f.y * a4.y;
      num[1][1] += f.y * a4.w;
      num[1][2] += f.y * b4.y;
      num[1][3] += f.y * b4.w;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (r0 + i < R)
        *reinterpret_cast<float4 *>(part_o +
                                    ((int64_t)part * rows_out + query_row(bi0, r0 + i, lgG, H, j)) * kD +
                                    16 * (l >> 2) + 4 * mp) =
            make_float4(num[i][0], num[i][1], num[i][2], num[i][3]);
  }
  if (pl.tc) griddep_wait();
}

// `ways` warps of a CTA per output row, each with every ways-th of its parts:
// rows x ways are to keep every SM busy where there are few rows.  Lane s of a
// warp holds the weights of its parts s, s + 32, ..
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(PrefixAttnArgs a, Plan pl, int ways,
                                                               const float *__restrict__ part_lse,
                                                               const float *__restrict__ part_o) {
  __shared__ float sh_m[kJoinWarps], sh_den[kJoinWarps];
  __shared__ float4 sh_o[kJoinWarps][32];
  const int H = (int)a.H, L = (int)a.L, rows = (int)a.B * L * H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int way = warp & (ways - 1);
  const int row = min(blockIdx.x * (kJoinWarps / ways) + warp / ways, rows - 1);
  const bool dup = (int)(blockIdx.x * (kJoinWarps / ways) + warp / ways) >= rows;
  const int bi = row / H, h = row - bi * H;
  // the parts of this row: np of the prefix, then those of its own tokens
  int np = pl.p_splits;
  if (pl.tc)
    np = tc_parts(pl, (h >> pl.lgG) * pl.tc_groups +
                          ((bi << pl.lgG) + (h & (pl.G - 1))) / pl.tc_rows);
  auto slot = [&](int s) { return (int64_t)(s < np ? s : pl.p_splits + s - np) * rows + row; };
  griddep_wait();
  griddep_launch_dependents();
  const int len = a.len[bi / L];
  const int parts = np + pl.o_splits, mine = parts > way ? (parts - way - 1) / ways + 1 : 0;
  // few parts: their outputs are read beside their weights, needed or not
  constexpr int kFew = 4;
  const bool few = mine <= kFew;
  float4 early[kFew];
  if (few) {
#pragma unroll
    for (int s = 0; s < kFew; ++s)
      if (s < mine) early[s] = reinterpret_cast<const float4 *>(part_o + slot(way + s * ways) * kD)[lane];
  }
  float M = -INFINITY, first = -INFINITY;
  bool nan = false;  // fmaxf passes over NaN, which the output must show
  for (int s = lane; s < mine; s += 32) {
    const float v = part_lse[slot(way + s * ways)];
    if (s == lane) first = v;
    M = fmaxf(M, v);
    nan |= v != v;
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  if (__any_sync(0xffffffffu, nan)) M = NAN;
  float den = 0.0f, o[4] = {};
  auto add = [&](float w, const float4 &v) {
    den += w;
    o[0] += w * v.x;
    o[1] += w * v.y;
    o[2] += w * v.z;
    o[3] += w * v.w;
  };
  if (M != -INFINITY)
    for (int s0 = 0; s0 < mine; s0 += 32) {
      const int at = s0 + lane;
      const float ls = s0 == 0 ? first : at < mine ? part_lse[slot(way + at * ways)] : -INFINITY;
      const float f = at < mine ? exp2f(ls - M) : 0.0f;
      if (few) {
#pragma unroll
        for (int s = 0; s < kFew; ++s) {
          const float w = __shfl_sync(0xffffffffu, f, s);
          if (w != 0.0f) add(w, early[s]);  // a part without weight writes no output
        }
        break;
      }
      // the parts with weight, four at a time
      uint32_t left = __ballot_sync(0xffffffffu, f != 0.0f);
      while (left) {
        float w[4];
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int s = left ? __ffs(left) - 1 : 0;
          w[i] = __shfl_sync(0xffffffffu, f, s);
          if (!left) w[i] = 0.0f;
          if (left) v[i] = reinterpret_cast<const float4 *>(part_o + slot(way + (s0 + s) * ways) * kD)[lane];
          left &= left - 1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (w[i] != 0.0f) add(w[i], v[i]);
      }
    }
  if (ways > 1) {  // the same for the whole grid
    if (lane == 0) {
      sh_m[warp] = M;
      sh_den[warp] = den;
    }
    sh_o[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    if (way != 0) return;
    float most = -INFINITY;
    nan = false;
    for (int w = 0; w < ways; ++w) {
      most = fmaxf(most, sh_m[warp + w]);
      nan |= sh_m[warp + w] != sh_m[warp + w];
    }
    M = nan ? NAN : most;
    den = o[0] = o[1] = o[2] = o[3] = 0.0f;
    for (int w = 0; w < ways; ++w) {
      if (sh_m[warp + w] == -INFINITY) continue;
      const float f = exp2f(sh_m[warp + w] - M);
      const float4 v = sh_o[warp + w][lane];
      den += f * sh_den[warp + w];
      o[0] += f * v.x;
      o[1] += f * v.y;
      o[2] += f * v.z;
      o[3] += f * v.w;
    }
  }
  if (dup || len < 0) return;
  // NaN scores give NaN; a row that sees nothing: zeros
  const float inv = den == 0.0f ? 0.0f : 1.0f / den;
  const uint2 w = make_uint2(pack_half2(o[0] * inv, o[1] * inv), pack_half2(o[2] * inv, o[3] * inv));
  reinterpret_cast<uint2 *>(a.out + (int64_t)row * kD)[lane] = w;
  if (a.lse && lane == 0)
    a.lse[row] = den == 0.0f ? -INFINITY : (M + log2f(den)) * 0.69314718055994531f;
}

// False where a count is past what the kernels' integers hold.
bool make_plan(Plan &p, int64_t B, int64_t L, int64_t H, int64_t Hkv, int64_t P, int64_t cap) {
  p = {};
  p.G = (int)(H / Hkv);
  while ((1 << p.lgG) < p.G) ++p.lgG;
  const int64_t most = 0x3fffffff;
  const int64_t R = B * L * p.G;
  p.tc = P > 0 && R >= kTcMinRows && Hkv * ((R + 15) / 16) * ((P + 15) / 16) >= kTcMinTiles;
  if (p.tc) {
    const int64_t tiles = (P + kTcTokens - 1) / kTcTokens, halves = (R + kTcTile - 1) / kTcTile;
    p.tc_rows = Hkv * halves * tiles <= kSms ? kTcTile : 2 * kTcTile;
    const int64_t groups = (R + p.tc_rows - 1) / p.tc_rows, units = Hkv * groups * tiles;
    if (units > most) return false;
    p.tc_groups = (int)groups;
    p.tc_tiles = (int)tiles;
    p.tc_units = (int)units;
    // as many CTAs as the longest run of units needs: fewer parts to join, and
    // SMs for the own tokens
    p.tc_run = (int)((units + kSms - 1) / kSms);
    p.tc_ctas = (int)((units + p.tc_run - 1) / p.tc_run);
    // the most CTAs whose runs meet one item's units
    p.p_splits = (int)min((int64_t)p.tc_ctas, (tiles + p.tc_run - 2) / p.tc_run + 1);
  } else if (P > 0) {
    const int64_t row_tiles = (R + kRows - 1) / kRows;
    p.row_warps = row_tiles >= 8 ? 8 : row_tiles >= 4 ? 4 : row_tiles >= 2 ? 2 : 1;
    p.p_groups = (int)((row_tiles + p.row_warps - 1) / p.row_warps);
    // One CTA an SM with few tokens each, two with more: four tiles a warp.
    const int64_t step = kTile * (kWarps / p.row_warps), base = Hkv * p.p_groups;
    int64_t s = max((kSms + base - 1) / base, min((2 * kSms + base - 1) / base, P / (4 * step)));
    s = max((int64_t)1, min(min(s, (int64_t)64), (P + step - 1) / step));
    p.p_len = (int)(((P + s - 1) / s + step - 1) / step * step);
    p.p_splits = (int)((P + p.p_len - 1) / p.p_len);
    if (p.p_splits * base > most) return false;
    p.p_ctas = (int)(p.p_splits * base);
  }
  p.o_tiles = (int)((L * p.G + kRows - 1) / kRows);
  if (cap > 0) {
    // One CTA an SM with few tokens each, four with more (two at a time: lengths
    // differ): three tiles a warp.  74 caches of 0 to 3001 tokens beside their prefix
    // 31.5 us (33.7 with two CTAs an SM and four tiles a warp), 128 of 0 to 1024 the same.
    const int64_t step = kTile * kWarps, base = B * Hkv * p.o_tiles;
    int64_t s = max((kSms + base - 1) / base, min((4 * kSms + base - 1) / base, cap / (3 * step)));
    s = max((int64_t)1, min(s, (cap + step - 1) / step));
    p.o_len = (int)(((cap + s - 1) / s + step - 1) / step * step);
    p.o_splits = (int)((cap + p.o_len - 1) / p.o_len);
    if (base * p.o_splits > most) return false;
    p.o_ctas = (int)(base * p.o_splits);
  }
  return p.p_ctas + p.o_ctas <= most;
}

}  // namespace pattn

bool prefix_attention_supported(int64_t B, int64_t L, int64_t H, int64_t Hkv, int64_t P,
                                int64_t cap) {
  if (B < 0 || L < 1 || Hkv < 1 || H < Hkv || H % Hkv != 0 || P < 0 || cap < 0) return false;
  const int64_t g = H / Hkv;
  if (g != 1 && g != 2 && g != 4 && g != 8) return false;
  const int64_t lim = (int64_t)1 << 30;
  if (B > lim || L > lim || H > 65535 || P > lim || cap > lim) return false;
  if (B * L > lim / H || B * Hkv > (int64_t)1 << 22) return false;
  if (B == 0) return true;
  pattn::Plan p;
  return pattn::make_plan(p, B, L, H, Hkv, P, cap);
}

int64_t prefix_attention_ws_bytes(int64_t B, int64_t L, int64_t H, int64_t Hkv, int64_t P,
                                  int64_t cap) {
  if (B == 0) return 0;
  pattn::Plan p;
  if (!pattn::make_plan(p, B, L, H, Hkv, P, cap)) return 0;
  const int64_t rows = (int64_t)(p.p_splits + p.o_splits) * B * L * H;
  return (rows + 3) / 4 * 16 + rows * pattn::kD * 4;
}

cudaError_t launch_prefix_attention(const PrefixAttnArgs &a, cudaStream_t st) {
  pattn::Plan p;
  if (!pattn::make_plan(p, a.B, a.L, a.H, a.Hkv, a.P, a.cap)) return cudaErrorInvalidValue;
  const int64_t out_rows = a.B * a.L * a.H;
  const int64_t rows = (int64_t)(p.p_splits + p.o_splits) * out_rows;
  float *lse = static_cast<float *>(a.ws);
  float *o = lse + (rows + 3) / 4 * 4;
  const int ctas = p.p_ctas + p.o_ctas;
  if (p.tc) {
    cudaError_t e = pattn::launch_prefix_tc(a, p, lse, o, st);
    if (e != cudaSuccess) return e;
  }
  if (ctas > 0) {
    // where no CTA has more than 8 rows, its second 8 are left out
    const int64_t most = (p.p_ctas > 0 ? a.B * a.L : a.L) * p.G;
    auto kern = most <= 8 ? (a.mode ? pattn::parts_kernel<1, 1> : pattn::parts_kernel<0, 1>)
                          : (a.mode ? pattn::parts_kernel<1, 2> : pattn::parts_kernel<0, 2>);
    const int smem = pattn::smem_bytes(a.mode, p.p_ctas > 0 ? p.row_warps : 1);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         pattn::smem_bytes(a.mode, pattn::kWarps));
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)ctas), dim3(pattn::kThreads), smem, st, true, a, p, lse, o);
    if (e != cudaSuccess) return e;
  }
  // 592 rows of 28 parts take 7.0 us with a warp each and 4.7 with four, 2048 rows of 17
  // parts 7.1 us with one and 9.5 with four
  int ways = 1;
  while (ways < pattn::kJoinWarps && out_rows * ways < 12 * pattn::kSms &&
         p.p_splits + p.o_splits > 2 * ways)
    ways *= 2;
  const int64_t per = pattn::kJoinWarps / ways;
  return launch_pdl(pattn::join_kernel, dim3((unsigned)((out_rows + per - 1) / per)),
                    dim3(pattn::kJoinWarps * 32), 0, st, true, a, p, ways, (const float *)lse,
                    (const float *)o);
}

}  // namespace bitnest
