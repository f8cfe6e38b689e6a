// Rotary positions, and the rows of a nested KV cache: written (rotated,
// packed) and read back.
//
// A rotary position turns pairs of a head's first `rot` values by the angle
// w = pos * theta_i:  (a, b) -> m (a cos w - b sin w, a sin w + b cos w).
// theta_i is held as a 64-bit fixed-point fraction of a turn per position
// (phase_i = theta_i / 2 pi * 2^64), so that pos * phase_i modulo 2^64 IS the
// angle modulo a turn: one integer multiplication, no error that grows with
// the position (2^-65 turns a position; an fp32 angle is off by 0.008 radians
// at position 131072), and negative positions turn the other way by
// themselves.  The top 32 bits become the argument of sincospif in [-1, 1).
#include "common.cuh"
#include "launch.h"
#include "nested_mma.cuh"

namespace bitnest {

namespace rows {

// m cos and m sin of the angle at `pos` (sign: +1, or -1 for the inverse turn)
__device__ __forceinline__ void turn(uint64_t phase, int32_t pos, float sign, float mag, float &c,
                                     float &s) {
  const uint64_t frac = phase * (uint64_t)(int64_t)pos;  // turns, modulo one
  // half turns in [-1, 1): 24 significant bits of the 32 kept, off by at most
  // 2^-25 half turns = 9.4e-8 radians
  const float half_turns = (float)(int32_t)(frac >> 32) * 4.656612873077393e-10f;  // 2^-31
  sincospif(half_turns, &s, &c);
  c *= mag;
  s *= mag * sign;
}

// Plain loads where the array may be written by the same kernel (rope in place), the
// read-only path elsewhere.
template <bool RO, typename U>
__device__ __forceinline__ U load(const U *p) {
  if constexpr (RO) return __ldg(p);
  return *p;
}

// N consecutive values of type T as fp32, by loads of up to 16 bytes.
template <bool RO, typename T, int N>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[N]) {
  constexpr int kBytes = sizeof(T) * N;
  if constexpr (sizeof(T) == 4) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const float4 f = load<RO>(reinterpret_cast<const float4 *>(p) + i);
        v[4 * i] = f.x;
        v[4 * i + 1] = f.y;
        v[4 * i + 2] = f.z;
        v[4 * i + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = load<RO>(p + i);
    }
  } else if constexpr (kBytes % 8 == 0) {
    uint32_t w[N / 2];
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
        const uint4 u = load<RO>(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const uint2 u = load<RO>(reinterpret_cast<const uint2 *>(p) + i);
        w[2 * i] = u.x;
        w[2 * i + 1] = u.y;
      }
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __half2float(p[i]);
  }
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[N]) {
  constexpr int kBytes = sizeof(T) * N;
  if constexpr (sizeof(T) == 4) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        reinterpret_cast<float4 *>(p)[i] =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = v[i];
    }
  } else if constexpr (kBytes % 8 == 0) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i)
        reinterpret_cast<uint4 *>(p)[i] =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        reinterpret_cast<uint2 *>(p)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = __float2half_rn(v[i]);
  }
}

// N values as they lie, where they are whole 16-byte pieces, and as fp32.
template <typename T, int N>
struct Raw {
  static constexpr int kPieces = (int)sizeof(T) * N / 16;
  uint4 w[kPieces];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + k] = __uint_as_float(u[k]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[k]));
          v[8 * i + 2 * k] = f.x;
          v[8 * i + 2 * k + 1] = f.y;
        }
      }
    }
  }
};

// ------------------------------------------------------------------- rope
// A thread owns V pairs of one token (2 V values: two runs of V in the halves
// layout, one run of 2 V of adjacent pairs) and goes over `per` heads with
// the same cosines and sines; the values behind `rot` are copied 2 V a thread.
// Every value is read, by plain loads, and written by one thread, so x may be y.
template <typename TX, typename TY, int V, bool PAIRS>
__global__ void __launch_bounds__(256) rope_kernel(
    const TX *x, int64_t x_token, int64_t x_head, TY *y, int64_t y_token, int64_t y_head,
    const int32_t *__restrict__ pos, const uint64_t *__restrict__ phase, float mag,
    float sign, int64_t M, int heads, int D, int rot, int per) {
  const int turned = rot / (2 * V);                            // units of a head that turn
  const int units = turned + (D - rot + 2 * V - 1) / (2 * V);  // and all of them
  const int groups = (heads + per - 1) / per;
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t token = id / (units * groups);
  if (token >= M) return;
  const int rest = (int)(id - token * (units * groups));
  const int hg = rest / units, u = rest - hg * units;
  const int h_end = min(heads, (hg + 1) * per);
  const TX *xp = x + token * x_token + hg * per * x_head;
  TY *yp = y + token * y_token + hg * per * y_head;
  if (u < turned) {
    float c[V], s[V];
    const int32_t p = pos[token];
#pragma unroll
    for (int i = 0; i < V; ++i) turn(phase[u * V + i], p, sign, mag, c[i], s[i]);
    auto turn_head = [&](float (&a)[V], float (&b)[V], TY *y) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float t = a[i] * c[i] - b[i] * s[i];
        b[i] = a[i] * s[i] + b[i] * c[i];
        a[i] = t;
      }
      if constexpr (PAIRS) {
        float v[2 * V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[2 * i] = a[i], v[2 * i + 1] = b[i];
        store_vec<TY, 2 * V>(y + 2 * V * u, v);
      } else {
        store_vec<TY, V>(y + V * u, a);
        store_vec<TY, V>(y + rot / 2 + V * u, b);
      }
    };
    if constexpr (V == 8) {
      // the loads of a few heads in flight together, as they lie (x may be y, but
      // a value is read and written by one thread only)
      constexpr int kBatch = sizeof(TX) == 4 ? 2 : 4;
      for (int h = hg * per; h < h_end; h += kBatch, xp += kBatch * x_head, yp += kBatch * y_head) {
        Raw<TX, V> lo[kBatch], hi[kBatch];
#pragma unroll
        for (int n = 0; n < kBatch; ++n)
          if (h + n < h_end) {
            lo[n].load(xp + n * x_head + (PAIRS ? 2 * V * u : V * u));
            hi[n].load(xp + n * x_head + (PAIRS ? 2 * V * u + V : rot / 2 + V * u));
          }
#pragma unroll
        for (int n = 0; n < kBatch; ++n)
          if (h + n < h_end) {
            float p[V], q[V];
            lo[n].get(p);
            hi[n].get(q);
            if constexpr (PAIRS) {
              float a[V], b[V];
#pragma unroll
              for (int i = 0; i < V / 2; ++i) {
                a[i] = p[2 * i], b[i] = p[2 * i + 1];
                a[V / 2 + i] = q[2 * i], b[V / 2 + i] = q[2 * i + 1];
              }
              turn_head(a, b, yp + n * y_head);
            } else {
              turn_head(p, q, yp + n * y_head);
            }
          }
      }
    } else {
#pragma unroll 2
      for (int h = hg * per; h < h_end; ++h, xp += x_head, yp += y_head) {
        float a[V], b[V];
        if constexpr (PAIRS) {
          float v[2 * V];
          load_vec<false, TX, 2 * V>(xp + 2 * V * u, v);
#pragma unroll
          for (int i = 0; i < V; ++i) a[i] = v[2 * i], b[i] = v[2 * i + 1];
        } else {
          load_vec<false, TX, V>(xp + V * u, a);
          load_vec<false, TX, V>(xp + rot / 2 + V * u, b);
        }
        turn_head(a, b, yp);
      }
    }
  } else {
    const int at = rot + (u - turned) * 2 * V;
    if constexpr (V == 8) {
      constexpr int kBatch = sizeof(TX) == 4 ? 2 : 4;
      for (int h = hg * per; h < h_end; h += kBatch, xp += kBatch * x_head, yp += kBatch * y_head) {
        Raw<TX, 2 * V> v[kBatch];
#pragma unroll
        for (int n = 0; n < kBatch; ++n)
          if (h + n < h_end) v[n].load(xp + n * x_head + at);
#pragma unroll
        for (int n = 0; n < kBatch; ++n)
          if (h + n < h_end) {
            float f[2 * V];
            v[n].get(f);
            store_vec<TY, 2 * V>(yp + n * y_head + at, f);
          }
      }
    } else {
      for (int h = hg * per; h < h_end; ++h, xp += x_head, yp += y_head) {
        if constexpr (V > 1) {
          // in the runs of the turned values, whose alignment was asked for
          constexpr int kRun = PAIRS ? 2 * V : V;
#pragma unroll
          for (int r = 0; r < 2 * V; r += kRun) {
            float v[kRun];
            load_vec<false, TX, kRun>(xp + at + r, v);
            store_vec<TY, kRun>(yp + at + r, v);
          }
        } else {
          for (int i = at; i < min(D, at + 2); ++i) {
            float v[1];
            load_vec<false, TX, 1>(xp + i, v);
            store_vec<TY, 1>(yp + i, v);
          }
        }
      }
    }
  }
}

constexpr int kMostHeads = 8;  // 8192 x 32 x 128 fp16: 27.9 us, 28.8 with 4, 39.8 with 2 (cosines), 31.2 with 16
template <typename TX, typename TY, int V>
cudaError_t launch_rope_v(const RopeArgs &a, cudaStream_t st) {
  const int64_t units = a.rot / (2 * V) + (a.D - a.rot + 2 * V - 1) / (2 * V);
  // Heads a thread goes over with one set of cosines and sines: as many as
  // leave two blocks of 256 threads for each SM, at most kMostHeads.
  int per = 1;
  while (per < kMostHeads && per < a.heads &&
         a.M * units * ((a.heads + 2 * per - 1) / (2 * per)) >= 2 * 148 * 256)
    per *= 2;
  const int64_t threads = a.M * units * ((a.heads + per - 1) / per);
  const int64_t blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto kern = a.pairs ? rope_kernel<TX, TY, V, true> : rope_kernel<TX, TY, V, false>;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, st, true,
                    static_cast<const TX *>(a.x), a.x_token, a.x_head, static_cast<TY *>(a.y),
                    a.y_token, a.y_head, a.pos, a.phase, a.mag, a.sign, a.M, (int)a.heads,
                    (int)a.D, (int)a.rot, per);
}

// 8 or 4 pairs a thread where the lengths, strides and addresses allow its
// loads and stores, else one.  No access is wider than a run of turned values or
// 16 bytes, and every one starts a multiple of V (2 V for pairs) values into a
// head: what `fits` asks of the addresses covers them all.
template <typename TX, typename TY>
cudaError_t launch_rope_t(const RopeArgs &a, cudaStream_t st) {
  auto fits = [&](int V) {
    const uintptr_t addr = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
    const int64_t strides = a.x_token | a.x_head | a.y_token | a.y_head;
    const int run = a.pairs ? 2 * V : V;  // values of one load
    const int bytes = run * (int)(sizeof(TX) > sizeof(TY) ? sizeof(TX) : sizeof(TY));
    return a.rot % (2 * V) == 0 && (a.D - a.rot) % (2 * V) == 0 && strides % (2 * V) == 0 &&
           addr % (uintptr_t)(bytes < 16 ? bytes : 16) == 0;
  };
  if (fits(8)) return launch_rope_v<TX, TY, 8>(a, st);
  if (fits(4)) return launch_rope_v<TX, TY, 4>(a, st);
  return launch_rope_v<TX, TY, 1>(a, st);
}

// ----------------------------------------------------------- cache rows
// A row is one token and one KV head, D = 128: 16 lanes, 8 values each.  Two
// rows to a warp.
constexpr int kD = 128;
constexpr int kRowLanes = 16;

__device__ __forceinline__ float max3_abs(float m, float a, float b) {
  return fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The low nibbles of eight words as the eight nibbles of one.
__device__ __forceinline__ uint32_t nibbles8(const uint32_t (&w)[8]) {
  uint32_t half[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t x = prmt(prmt(w[4 * h], w[4 * h + 1], 0x0040), prmt(w[4 * h + 2], w[4 * h + 3], 0x0040), 0x5410);
    half[h] = (x & 0x000F000Fu) | ((x >> 4) & 0x00F000F0u);  // bytes 0 and 2
  }
  return prmt(half[0], half[1], 0x6420);
}

// The packer's rule on 8 values of a row that are exact in fp16 (see
// pack_weights_kernel): s = fp16(max / 7), t = RN(x / s), q = rne(t),
// r = clamp(rne(16 (t - q)), -8, 7); nibbles q + 8 and r + 8.  |t| <= 7.01
// unless s is subnormal in fp16 and was rounded down; then q is clamped to
// -8 .. 7 as well.
//
// No division: T = 16 t is x 16 rcp(s), rounded to a multiple of 2^-13.  With
// x = X 2^a, s = S 2^b (X, S integers below 2^11) the exact T is off a half
// integer, where a rounding changes, by |32 X 2^(a-b) - (2 k + 1) S| / 2 S: by
// nothing or by 1 / 2 S > 2.4e-4 at least (for a - b < -5 as well: T <= 1/2
// then, and X < 2 S).  rcp is off by 2^-23 at most, so where |t| <= 7.25 the
// product is off by 2.2e-5: the rounding to 2^-13 gives the half integers
// exactly, and moves nothing else across one or onto one.
// Adding 1.5 * 2^23 rounds to an integer, 1.5 * 2^27 to a multiple of 16, whose
// two's complement is in the low bits; the codes' offset 8 flips a nibble's top
// bit.
__device__ __forceinline__ void pack8(const float (&x)[8], float m, float s, uint32_t &hi,
                                      uint32_t &lo) {
  constexpr float kInt = 12582912.0f, kSixteen = 201326592.0f;  // 1.5 * 2^23, 1.5 * 2^27
  constexpr float kGrid = 1536.0f;                              // 1.5 * 2^10: to 2^-13
  const float rs = s == 0.0f ? 0.0f : rcp_approx(s) * 16.0f;
  uint32_t qb[8], rb[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float t[2], q[2], u[2];
    f32x2_mul(t[0], t[1], x[i], x[i + 1], rs, rs);
    f32x2_add(t[0], t[1], t[0], t[1], kGrid, kGrid);
    f32x2_sub(t[0], t[1], t[0], t[1], kGrid, kGrid);
    f32x2_add(q[0], q[1], t[0], t[1], kSixteen, kSixteen);
    qb[i] = __float_as_uint(q[0]);
    qb[i + 1] = __float_as_uint(q[1]);
    f32x2_sub(q[0], q[1], q[0], q[1], kSixteen, kSixteen);
    f32x2_sub(u[0], u[1], t[0], t[1], q[0], q[1]);  // exact, |u| <= 8
    f32x2_add(u[0], u[1], u[0], u[1], kInt, kInt);
    rb[i] = __float_as_uint(fminf(u[0], kInt + 7.0f));
    rb[i + 1] = __float_as_uint(fminf(u[1], kInt + 7.0f));
  }
  if (m * rs > 16.0f * 7.25f) {  // a subnormal scale
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = __fdiv_rn(x[i], s);
      const float q = fmaxf(-8.0f, fminf(7.0f, rintf(t)));
      const float r = fmaxf(-8.0f, fminf(7.0f, rintf(__fmul_rn(16.0f, __fsub_rn(t, q)))));
      qb[i] = __float_as_uint(__fadd_rn(q, kInt));
      rb[i] = __float_as_uint(__fadd_rn(r, kInt));
    }
  }
  hi = nibbles8(qb) ^ 0x88888888u;  // column i in nibble i: byte i / 2, low nibble first
  lo = nibbles8(rb) ^ 0x88888888u;
}

__device__ __forceinline__ void round_half8(float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 f = __half22float2(__floats2half2_rn(v[i], v[i + 1]));
    v[i] = f.x;
    v[i + 1] = f.y;
  }
}

// One 16-lane group per token (of 16 in a block) and `per` heads (blockIdx.z);
// blockIdx.y = 0: keys, 1: values.  A lane has two runs of four columns, at c0
// and c1: the two of its four pairs in the halves layout, neighbours elsewhere.
// A batch of heads is loaded together.
//
// Bound: instructions (16384 x 8 fp16 rows are 101 MB, 15 us to move, and take 34: 23.3 M
// of them, issue slots 58 % and the ALU pipe 62 % busy): hence packed arithmetic, nibbles gathered by byte permutations, one reciprocal a
// row, and 32-bit indexes up to the row's.
constexpr int kBatch = 4;
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a, int per) {
  const int lane = threadIdx.x & (kRowLanes - 1);
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t token = blockIdx.x * 16u + threadIdx.x / kRowLanes;  // b * L + i
  const bool values = blockIdx.y != 0;
  // whole warps run on: the shuffles below need every lane
  bool live = token < (uint32_t)(a.B * a.L);
  int64_t row0 = 0;
  if (live) {
    const uint32_t b = token / (uint32_t)a.L, i = token - b * (uint32_t)a.L;
    const int64_t t = (int64_t)a.start[b] + i;
    live = t >= 0 && t < a.cap && (!a.count || (int)i < a.count[b]);
    row0 = (b * a.cap + t) * a.Hkv;
  }
  const int hg = blockIdx.z;
  const int rot = values || !a.phase ? 0 : (int)a.rot;
  const bool turning = 8 * lane < rot;
  const bool apart = !PAIRS && turning;
  const int c0 = apart ? 4 * lane : 8 * lane, c1 = apart ? rot / 2 + 4 * lane : 8 * lane + 4;
  float c[4], s[4];
  if (turning && live) {
    const int32_t p = a.pos[token];
#pragma unroll
    for (int i = 0; i < 4; ++i) turn(a.phase[4 * lane + i], p, 1.0f, a.mag, c[i], s[i]);
  }
  const T *src = static_cast<const T *>(values ? a.v : a.k) +
                 (live ? token * (values ? a.v_token : a.k_token) : 0);
  uint8_t *hi = values ? a.cache.v_hi : a.cache.k_hi;
  uint8_t *lo = values ? a.cache.v_lo : a.cache.k_lo;
  uint16_t *sc = values ? a.cache.v_scale : a.cache.k_scale;
  const int h_end = min((int)a.Hkv, (hg + 1) * per);
  for (int h = hg * per; h < h_end; h += kBatch) {
    float v[kBatch][8];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      if (live && h + n < h_end) {
        const T *p = src + (int64_t)(h + n) * kD;
        float x[4], y[4];
        load_vec<true, T, 4>(p + c0, x);
        load_vec<true, T, 4>(p + c1, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[n][i] = x[i], v[n][4 + i] = y[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[n][i] = 0.0f;
      }
    }
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      float(&x)[8] = v[n];
      if (turning)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float &p = x[PAIRS ? 2 * i : i], &q = x[PAIRS ? 2 * i + 1 : 4 + i];
          const float t = p * c[i] - q * s[i];
          q = p * s[i] + q * c[i];
          p = t;
        }
      // to fp16 first, as bitnest_rope's output is: the same bits as turning and
      // packing in two calls
      if (sizeof(T) == 4 || turning) round_half8(x);
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; i += 2) m = max3_abs(m, x[i], x[i + 1]);
#pragma unroll
      for (int o = kRowLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      // fp16(m / 7): m / 7 is never within 2^-4 steps of the middle of two fp16
      // values (7 (2 k + 1) is odd), the product within 2^-23 of it
      const __half sh = __float2half_rn(m * 0.14285714285714286f);
      uint32_t h4, l4;
      pack8(x, m, __half2float(sh), h4, l4);
      if (live && h + n < h_end) {
        const int64_t row = row0 + h + n;
        uint8_t *ph = hi + row * (kD / 2), *pl = lo + row * (kD / 2);
        if (apart) {
          *reinterpret_cast<uint16_t *>(ph + c0 / 2) = (uint16_t)h4;
          *reinterpret_cast<uint16_t *>(ph + c1 / 2) = (uint16_t)(h4 >> 16);
          *reinterpret_cast<uint16_t *>(pl + c0 / 2) = (uint16_t)l4;
          *reinterpret_cast<uint16_t *>(pl + c1 / 2) = (uint16_t)(l4 >> 16);
        } else {
          *reinterpret_cast<uint32_t *>(ph + c0 / 2) = h4;
          *reinterpret_cast<uint32_t *>(pl + c0 / 2) = l4;
        }
        if (lane == 0) sc[row] = __half_as_ushort(sh);
      }
    }
  }
}

// 16 lanes a row, 8 values (4 bytes of each plane) a lane; a token (of 16 in a
// block) and four heads (blockIdx.z) a thread; blockIdx.y as above.  The codes
// are exact in fp16 (in sixteenths for the target), so one fp16 product with
// the scale rounds once.
constexpr int kReadRows = 4;
template <int MODE>
__global__ void __launch_bounds__(256) kv_read_kernel(ReadArgs a) {
  const int lane = threadIdx.x & (kRowLanes - 1);
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t token = blockIdx.x * 16u + threadIdx.x / kRowLanes;
  if (token >= (uint32_t)(a.B * a.L)) return;
  const uint32_t b = token / (uint32_t)a.L;
  const int64_t t = (a.start ? (int64_t)a.start[b] : 0) + (token - b * (uint32_t)a.L);
  const bool in = t >= 0 && t < a.cap;  // rows outside the cache read as zeros
  const bool values = blockIdx.y != 0;
  const int j0 = blockIdx.z * kReadRows, heads = min((int)a.Hkv - j0, kReadRows);
  const int64_t row = (b * a.cap + t) * a.Hkv + j0;
  const uint32_t *hi = reinterpret_cast<const uint32_t *>((values ? a.cache.v_hi : a.cache.k_hi) + row * (kD / 2)) + lane;
  const uint32_t *lo = reinterpret_cast<const uint32_t *>((values ? a.cache.v_lo : a.cache.k_lo) + row * (kD / 2)) + lane;
  const uint16_t *sc = (values ? a.cache.v_scale : a.cache.k_scale) + row;
  uint4 *out = reinterpret_cast<uint4 *>((values ? a.v : a.k) + ((int64_t)token * a.Hkv + j0) * kD) + lane;
  uint32_t h[kReadRows], l[kReadRows];
  uint16_t s[kReadRows];
#pragma unroll
  for (int n = 0; n < kReadRows; ++n) {
    h[n] = l[n] = 0x88888888u;
    s[n] = 0;
    if (in && n < heads) {
      h[n] = hi[n * (kD / 8)];
      if (MODE) l[n] = lo[n * (kD / 8)];
      s[n] = sc[n];
    }
  }
#pragma unroll
  for (int n = 0; n < kReadRows; ++n) {
    if (n >= heads) break;
    uint32_t ev, od, w[4];
    nested::codes<MODE>(h[n], l[n], ev, od);
    const __half2 scale = __half2half2(__ushort_as_half(s[n]));
    // 0x6400 | u is 1024 + u: times 1/16 and less (1024 + 136) / 16, exact
    const __half2 unit = __float2half2_rn(MODE ? 0.0625f : 1.0f);
    const __half2 offset = __float2half2_rn(MODE ? -72.5f : -1032.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = (prmt(ev, od, (uint32_t)i | ((uint32_t)(i + 4) << 8)) & 0x00FF00FFu) | 0x64006400u;
      const __half2 v = __hmul2(__hfma2(*reinterpret_cast<const __half2 *>(&u), unit, offset), scale);
      w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    out[n * (kD / 8)] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace rows

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st) {
  if (a.x_type == 0)
    return a.y_type == 0 ? rows::launch_rope_t<__half, __half>(a, st)
                         : rows::launch_rope_t<__half, float>(a, st);
  return a.y_type == 0 ? rows::launch_rope_t<float, __half>(a, st)
                       : rows::launch_rope_t<float, float>(a, st);
}

cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t st) {
  // Heads that a 16-lane group goes over with one set of cosines and sines:
  // as many as leave four blocks for each SM, at most 8, and at least what the
  // grid's third dimension asks for.
  const int64_t blocks = (a.B * a.L + 15) / 16;
  int per = 1;
  while (per < a.Hkv && ((per < 8 && 2 * blocks * ((a.Hkv + 2 * per - 1) / (2 * per)) >= 4 * 148) ||
                         (a.Hkv + per - 1) / per > 65535))
    per *= 2;
  const dim3 grid((unsigned)blocks, 2, (unsigned)((a.Hkv + per - 1) / per));
  auto kern = a.type == 0 ? (a.pairs ? rows::kv_append_kernel<__half, true>
                                     : rows::kv_append_kernel<__half, false>)
                          : (a.pairs ? rows::kv_append_kernel<float, true>
                                     : rows::kv_append_kernel<float, false>);
  return launch_pdl(kern, grid, dim3(256), 0, st, true, a, per);
}

cudaError_t launch_kv_read(const ReadArgs &a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.B * a.L + 15) / 16), 2,
                  (unsigned)((a.Hkv + rows::kReadRows - 1) / rows::kReadRows));
  auto kern = a.mode ? rows::kv_read_kernel<1> : rows::kv_read_kernel<0>;
  return launch_pdl(kern, grid, dim3(256), 0, st, true, a);
}

}  // namespace bitnest
