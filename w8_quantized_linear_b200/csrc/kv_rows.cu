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

// N consecutive values of type T as fp32, by loads of up to 16 bytes.
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[N]) {
  constexpr int kBytes = sizeof(T) * N;
  if constexpr (sizeof(T) == 4) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(p) + i);
        v[4 * i] = f.x;
        v[4 * i + 1] = f.y;
        v[4 * i + 2] = f.z;
        v[4 * i + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __ldg(p + i);
    }
  } else if constexpr (kBytes % 8 == 0) {
    uint32_t w[N / 2];
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p) + i);
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

// ------------------------------------------------------------------- rope
// A thread owns V pairs of one token (2 V values: two runs of V in the halves
// layout, one run of 2 V of adjacent pairs) and goes over `per` heads with
// the same cosines and sines; the values behind `rot` are copied in runs of
// 2 V.  Every value is read and written by one thread, so x may be y.
template <typename TX, typename TY, int V, bool PAIRS>
__global__ void __launch_bounds__(256) rope_kernel(
    const TX *__restrict__ x, int64_t x_token, int64_t x_head, TY *__restrict__ y, int64_t y_token,
    int64_t y_head, const int32_t *__restrict__ pos, const uint64_t *__restrict__ phase, float mag,
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
#pragma unroll 2
    for (int h = hg * per; h < h_end; ++h, xp += x_head, yp += y_head) {
      if constexpr (PAIRS) {
        float v[2 * V];
        load_vec<TX, 2 * V>(xp + 2 * V * u, v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float a = v[2 * i], b = v[2 * i + 1];
          v[2 * i] = a * c[i] - b * s[i];
          v[2 * i + 1] = a * s[i] + b * c[i];
        }
        store_vec<TY, 2 * V>(yp + 2 * V * u, v);
      } else {
        float a[V], b[V];
        load_vec<TX, V>(xp + V * u, a);
        load_vec<TX, V>(xp + rot / 2 + V * u, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float t = a[i] * c[i] - b[i] * s[i];
          b[i] = a[i] * s[i] + b[i] * c[i];
          a[i] = t;
        }
        store_vec<TY, V>(yp + V * u, a);
        store_vec<TY, V>(yp + rot / 2 + V * u, b);
      }
    }
  } else {
    const int at = rot + (u - turned) * 2 * V;
    for (int h = hg * per; h < h_end; ++h, xp += x_head, yp += y_head) {
      if constexpr (V > 1) {
        float v[2 * V];
        load_vec<TX, 2 * V>(xp + at, v);
        store_vec<TY, 2 * V>(yp + at, v);
      } else {
        for (int i = at; i < min(D, at + 2); ++i) {
          float v[1];
          load_vec<TX, 1>(xp + i, v);
          store_vec<TY, 1>(yp + i, v);
        }
      }
    }
  }
}

template <typename TX, typename TY, int V>
cudaError_t launch_rope_v(const RopeArgs &a, cudaStream_t st) {
  const int64_t units = a.rot / (2 * V) + (a.D - a.rot + 2 * V - 1) / (2 * V);
  // Heads a thread goes over with one set of cosines and sines: as many as
  // leave two blocks of 256 threads for each SM, at most 8.
  int per = 1;
  while (per < 8 && per < a.heads &&
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
// loads and stores, else one.
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

// max |v| over the 16 lanes of a row
__device__ __forceinline__ float row_max(float m) {
#pragma unroll
  for (int o = kRowLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The packer's rule on 8 values of a row that are exact in fp16 (see
// pack_weights_kernel): s = fp16(max / 7), t = RN(x / s), q = rne(t),
// r = clamp(rne(16 (t - q)), -8, 7); nibbles q + 8 and r + 8.  |t| <= 7.01
// unless s is subnormal in fp16 and was rounded down; then q is clamped to
// -8 .. 7 as well.
//
// The division is done as RN(x RN(1 / s)): where |t| <= 7.25 that is within
// 1.1e-6 of x / s and RN(x / s) within 2.4e-7, so 16 t is known to 2.2e-5 and
// both nibbles are the same unless 16 t lies within 2^-15 of a half-integer
// (r) or of 8 mod 16 (q); only such a value pays for the divisions.
__device__ __forceinline__ void pack8(const float (&x)[8], float m, float s, uint32_t &hi,
                                      uint32_t &lo) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer
  constexpr float kNear = 3.0517578125e-05f;
  const float rs = s == 0.0f ? 0.0f : __frcp_rn(s);
  hi = lo = 0;
  bool near = m * rs > 7.25f;
  uint32_t qb[8], rb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __fmul_rn(x[i], rs);
    const float q = __fsub_rn(__fadd_rn(t, kRound), kRound);
    const float u = __fmul_rn(16.0f, __fsub_rn(t, q));  // exact, |u| <= 8
    const float ur = __fadd_rn(u, kRound);
    const float r = __fsub_rn(ur, kRound);
    near |= fabsf(__fsub_rn(u, r)) > 0.5f - kNear || fabsf(u) > 8.0f - kNear;
    qb[i] = __float_as_uint(__fadd_rn(q, kRound + 8.0f));
    rb[i] = __float_as_uint(__fadd_rn(fminf(r, 7.0f), kRound + 8.0f));
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float q = 0.0f, r = 0.0f;
      if (s != 0.0f) {
        const float t = __fdiv_rn(x[i], s);
        q = fmaxf(-8.0f, fminf(7.0f, rintf(t)));
        r = fmaxf(-8.0f, fminf(7.0f, rintf(__fmul_rn(16.0f, __fsub_rn(t, q)))));
      }
      qb[i] = __float_as_uint(__fadd_rn(q, kRound + 8.0f));
      rb[i] = __float_as_uint(__fadd_rn(r, kRound + 8.0f));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // column i in nibble i: byte i / 2, low nibble first
    hi |= (qb[i] & 15u) << (4 * i);
    lo |= (rb[i] & 15u) << (4 * i);
  }
}

__device__ __forceinline__ void round_half8(float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __half2float(__float2half_rn(v[i]));
}

// One 16-lane group per (token, `per` heads), blockIdx.y = 0: keys, 1: values.
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a, int per) {
  const int lane = threadIdx.x & (kRowLanes - 1);
  const int64_t id = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) / kRowLanes;
  const int groups = ((int)a.Hkv + per - 1) / per;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t token = id / groups;  // b * L + i
  const bool values = blockIdx.y != 0;
  // whole warps run on: the shuffles below need every lane
  bool live = token < a.B * a.L;
  int64_t row0 = 0;
  if (live) {
    const int64_t b = token / a.L, i = token - b * a.L;
    const int64_t t = (int64_t)a.start[b] + i;
    live = t >= 0 && t < a.cap && (!a.count || i < a.count[b]);
    row0 = (b * a.cap + t) * a.Hkv;
  }
  const int hg = (int)(id - token * groups);
  float c[8], s[8];
  const bool turning = !values && a.phase != nullptr && 8 * lane < a.rot;
  const int half_lanes = (int)a.rot / 16;  // lanes of a half of the turned values
  if (turning && live) {
    const int32_t p = a.pos[token];
#pragma unroll
    for (int i = 0; i < (PAIRS ? 4 : 8); ++i) {
      const int pair = PAIRS ? 4 * lane + i : 8 * (lane < half_lanes ? lane : lane - half_lanes) + i;
      turn(a.phase[pair], p, 1.0f, a.mag, c[i], s[i]);
    }
  }
  const T *src = static_cast<const T *>(values ? a.v : a.k) +
                 (live ? token * (values ? a.v_token : a.k_token) : 0) + 8 * lane;
  uint8_t *hi = values ? a.cache.v_hi : a.cache.k_hi;
  uint8_t *lo = values ? a.cache.v_lo : a.cache.k_lo;
  uint16_t *sc = values ? a.cache.v_scale : a.cache.k_scale;
  for (int n = 0; n < per; ++n) {
    const int j = hg * per + n;
    const bool ok = live && j < a.Hkv;
    float v[8] = {};
    if (ok) load_vec<T, 8>(src + (int64_t)j * kD, v);
    if (a.phase != nullptr && !values) {  // the same for the whole block
      if constexpr (PAIRS) {
        if (turning)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = v[2 * i], y = v[2 * i + 1];
            v[2 * i] = x * c[i] - y * s[i];
            v[2 * i + 1] = x * s[i] + y * c[i];
          }
      } else {
        // the other of each pair sits half_lanes further
        const int other = (threadIdx.x & 16) |
                          (lane < half_lanes ? lane + half_lanes : turning ? lane - half_lanes : lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = __shfl_sync(0xffffffffu, v[i], other);
          if (turning) v[i] = lane < half_lanes ? v[i] * c[i] - w * s[i] : w * s[i] + v[i] * c[i];
        }
      }
    }
    // to fp16 first, as bitnest_rope's output is: the same bits as turning and
    // packing in two calls
    round_half8(v);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    m = row_max(m);
    const __half sh = __float2half_rn(__fdiv_rn(m, 7.0f));
    uint32_t h4, l4;
    pack8(v, m, __half2float(sh), h4, l4);
    if (ok) {
      const int64_t row = row0 + j;
      reinterpret_cast<uint32_t *>(hi + row * (kD / 2))[lane] = h4;
      reinterpret_cast<uint32_t *>(lo + row * (kD / 2))[lane] = l4;
      if (lane == 0) sc[row] = __half_as_ushort(sh);
    }
  }
}

// 16 lanes a row, 8 values (4 bytes of each plane) a lane; blockIdx.y as above.
template <int MODE>
__global__ void __launch_bounds__(256) kv_read_kernel(ReadArgs a) {
  const int lane = threadIdx.x & (kRowLanes - 1);
  const int64_t id = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) / kRowLanes;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t token = id / a.Hkv;
  if (token >= a.B * a.L) return;
  const int64_t b = token / a.L, i = token - b * a.L;
  const int64_t t = (a.start ? (int64_t)a.start[b] : 0) + i;
  const bool values = blockIdx.y != 0;
  uint16_t *out = (values ? a.v : a.k) + id * kD + 8 * lane;
  float v[8] = {};
  if (t >= 0 && t < a.cap) {  // rows outside the cache read as zeros
    const int64_t row = (b * a.cap + t) * a.Hkv + (id - token * a.Hkv);
    const uint32_t h =
        reinterpret_cast<const uint32_t *>((values ? a.cache.v_hi : a.cache.k_hi) + row * (kD / 2))[lane];
    uint32_t l = 0;
    if (MODE)
      l = reinterpret_cast<const uint32_t *>((values ? a.cache.v_lo : a.cache.k_lo) + row * (kD / 2))[lane];
    float s = __half2float(__ushort_as_half((values ? a.cache.v_scale : a.cache.k_scale)[row]));
    if (MODE) s *= 0.0625f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int q = (int)((h >> (4 * c)) & 15u);
      const int u = MODE ? 16 * q + (int)((l >> (4 * c)) & 15u) - 136 : q - 8;
      v[c] = (float)u * s;
    }
  }
  store_vec<__half, 8>(reinterpret_cast<__half *>(out), v);
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
  // as many as leave four blocks for each SM, at most 8.
  int per = 1;
  while (per < 8 && per < a.Hkv &&
         2 * a.B * a.L * ((a.Hkv + 2 * per - 1) / (2 * per)) * rows::kRowLanes >= 4 * 148 * 256)
    per *= 2;
  const int64_t threads = a.B * a.L * ((a.Hkv + per - 1) / per) * rows::kRowLanes;
  const int64_t blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks, 2);
  auto kern = a.type == 0 ? (a.pairs ? rows::kv_append_kernel<__half, true>
                                     : rows::kv_append_kernel<__half, false>)
                          : (a.pairs ? rows::kv_append_kernel<float, true>
                                     : rows::kv_append_kernel<float, false>);
  return launch_pdl(kern, grid, dim3(256), 0, st, true, a, per);
}

cudaError_t launch_kv_read(const ReadArgs &a, cudaStream_t st) {
  const int64_t blocks = (a.B * a.L * a.Hkv * rows::kRowLanes + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto kern = a.mode ? rows::kv_read_kernel<1> : rows::kv_read_kernel<0>;
  return launch_pdl(kern, dim3((unsigned)blocks, 2), dim3(256), 0, st, true, a);
}

}  // namespace bitnest
