// C ABI of rotary positions and of the nested KV cache's serving operators:
// host-side argument checks and dispatch.  The contract of each entry point
// is in include/bitnest.h.
#include <math.h>
#include <stdint.h>

#include "bitnest.h"
#include "common.cuh"
#include "launch.h"

using namespace bitnest;

namespace {

bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? BITNEST_OK : BITNEST_ERR_CUDA; }

constexpr int64_t kMost = (int64_t)1 << 30;  // tokens, rows of a call

// The planes that `mode` reads (both: a call that writes them all).
int check_planes(const bitnest_kv_cache *c, bool k, bool v, bool lo) {
  if (!c) return BITNEST_ERR_INVALID_ARG;
  const void *p[6] = {k ? c->k_hi : nullptr, k && lo ? c->k_lo : nullptr, k ? c->k_scale : nullptr,
                      v ? c->v_hi : nullptr, v && lo ? c->v_lo : nullptr, v ? c->v_scale : nullptr};
  const bool need[6] = {k, k && lo, k, v, v && lo, v};
  for (int i = 0; i < 6; ++i)
    if (need[i] && !p[i]) return BITNEST_ERR_INVALID_ARG;
  for (int i = 0; i < 6; ++i)
    if (need[i] && misaligned(p[i])) return BITNEST_ERR_MISALIGNED;
  return BITNEST_OK;
}

KvPlanes planes(const bitnest_kv_cache *c, bool lo = true) {
  if (!c) return KvPlanes{};
  return KvPlanes{c->k_hi, lo ? c->k_lo : nullptr, c->k_scale,
                  c->v_hi, lo ? c->v_lo : nullptr, c->v_scale};
}

bool cache_shape_ok(int64_t B, int64_t cap, int64_t Hkv) {
  return B >= 0 && cap >= 0 && cap <= kMost && Hkv >= 1 && Hkv <= 65535 && B <= kMost &&
         (B == 0 || cap == 0 || B * Hkv <= ((int64_t)1 << 46) / cap);
}

bool heads_ok(int64_t H, int64_t Hkv) {
  if (Hkv < 1 || H < Hkv || H > 65535 || H % Hkv != 0) return false;
  const int64_t g = H / Hkv;
  return g == 1 || g == 2 || g == 4 || g == 8;
}

}  // namespace

extern "C" {

int bitnest_rope_phases(int64_t rot, double base, int scaling, double factor, double low,
                        double high, int64_t trained, uint64_t *phase, float *magnitude) {
  if (rot < 2 || rot % 2 != 0 || rot > 65536) return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (!phase || !magnitude || !(base > 1.0) || !isfinite(base)) return BITNEST_ERR_INVALID_ARG;
  if (scaling < BITNEST_ROPE_PLAIN || scaling > BITNEST_ROPE_YARN) return BITNEST_ERR_INVALID_ARG;
  if (scaling != BITNEST_ROPE_PLAIN && !(factor >= 1.0 && isfinite(factor)))
    return BITNEST_ERR_INVALID_ARG;
  const bool spans = scaling == BITNEST_ROPE_BANDS || scaling == BITNEST_ROPE_YARN;
  if (spans && !(low > 0.0 && high > low && isfinite(high) && trained > 0))
    return BITNEST_ERR_INVALID_ARG;
  if (scaling == BITNEST_ROPE_NTK) {
    if (rot == 2) return BITNEST_ERR_UNSUPPORTED_SHAPE;  // its exponent rot / (rot - 2)
    base *= pow(factor, (double)rot / (double)(rot - 2));
  }
  const double turn = 6.283185307179586;
  double from = 0.0, to = 0.0;
  if (scaling == BITNEST_ROPE_YARN) {
    // the pair that makes `t` turns over the trained length
    auto pair = [&](double t) {
      return (double)rot * log((double)trained / (turn * t)) / (2.0 * log(base));
    };
    from = fmax(0.0, floor(pair(high)));
    to = fmin((double)(rot - 1), ceil(pair(low)));
  }
  for (int64_t i = 0; i < rot / 2; ++i) {
    double theta = pow(base, -2.0 * (double)i / (double)rot);
    if (scaling == BITNEST_ROPE_LINEAR) {
      theta /= factor;
    } else if (scaling == BITNEST_ROPE_BANDS) {
      const double t = fmin(1.0, fmax(0.0, ((double)trained * theta / turn - low) / (high - low)));
      theta *= t + (1.0 - t) / factor;
    } else if (scaling == BITNEST_ROPE_YARN) {
      const double r = fmin(1.0, fmax(0.0, ((double)i - from) / fmax(to - from, 1e-3)));
      theta *= 1.0 - r + r / factor;
    }
    // theta / 2 pi < 1/2 turn: the product stays below 2^63
    phase[i] = (uint64_t)llrint(theta / turn * 18446744073709551616.0);
  }
  *magnitude = scaling == BITNEST_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return BITNEST_OK;
}

int bitnest_rope(const void *x, int x_type, int64_t x_token, int64_t x_head, const int32_t *pos,
                 const uint64_t *phase, float magnitude, int64_t M, int64_t heads, int64_t D,
                 int64_t rot, int layout, int inverse, void *y, int y_type, int64_t y_token,
                 int64_t y_head, void *stream) {
  if (x_type != BITNEST_F16 && x_type != BITNEST_F32) return BITNEST_ERR_INVALID_ARG;
  if (y_type != BITNEST_F16 && y_type != BITNEST_F32) return BITNEST_ERR_INVALID_ARG;
  if (layout != BITNEST_ROPE_HALF && layout != BITNEST_ROPE_PAIRS) return BITNEST_ERR_INVALID_ARG;
  if (M < 0 || heads < 0 || D < 2 || D > 65536 || rot < 2 || rot > D || rot % 2 != 0)
    return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (heads > 65535 || M > kMost || M * heads > ((int64_t)1 << 46) / D)
    return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (M == 0 || heads == 0) return BITNEST_OK;
  // rows of y must not lie on one another
  const int64_t far = (int64_t)1 << 44;
  if (x_head < 0 || x_token < 0 || y_head < 0 || y_token < 0 || x_head > far || x_token > far ||
      y_head > far || y_token > far)
    return BITNEST_ERR_UNSUPPORTED_SHAPE;
  const bool by_token = (heads == 1 || y_head >= D) && (M == 1 || y_token >= (heads - 1) * y_head + D);
  const bool by_head = (M == 1 || y_token >= D) && (heads == 1 || y_head >= (M - 1) * y_token + D);
  if (!by_token && !by_head) return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (!x || !y || !pos || !phase) return BITNEST_ERR_INVALID_ARG;
  if (x == y && (x_type != y_type || (M > 1 && x_token != y_token) || (heads > 1 && x_head != y_head)))
    return BITNEST_ERR_INVALID_ARG;  // in place only onto itself
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ya = reinterpret_cast<uintptr_t>(y);
  if (xa % (x_type ? 4 : 2) || ya % (y_type ? 4 : 2) || reinterpret_cast<uintptr_t>(pos) % 4 ||
      reinterpret_cast<uintptr_t>(phase) % 8)
    return BITNEST_ERR_MISALIGNED;
  RopeArgs a{x, x_type, x_token, x_head, y, y_type, y_token, y_head, pos, phase, magnitude,
             inverse ? -1.0f : 1.0f, M, heads, D, rot, layout == BITNEST_ROPE_PAIRS};
  return cuda_status(launch_rope(a, (cudaStream_t)stream));
}

int bitnest_kv_append(const void *k, int64_t k_token, const void *v, int64_t v_token, int type,
                      int64_t B, int64_t L, int64_t Hkv, const int32_t *start,
                      const int32_t *count, const int32_t *pos, const uint64_t *phase,
                      float magnitude, int64_t rot, int layout, const bitnest_kv_cache *cache,
                      int64_t cap, void *stream) {
  if (type != BITNEST_F16 && type != BITNEST_F32) return BITNEST_ERR_INVALID_ARG;
  if (layout != BITNEST_ROPE_HALF && layout != BITNEST_ROPE_PAIRS) return BITNEST_ERR_INVALID_ARG;
  if (!cache_shape_ok(B, cap, Hkv) || L < 0 || L > kMost || (B > 0 && L > kMost / B) ||
      B * L > ((int64_t)1 << 38) / Hkv)
    return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (phase && (rot < 16 || rot > 128 || rot % 16 != 0)) return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (B == 0 || L == 0 || cap == 0) return BITNEST_OK;
  if (k_token < Hkv * 128 || v_token < Hkv * 128) return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (!k || !v || !start || (phase && !pos)) return BITNEST_ERR_INVALID_ARG;
  const int s = check_planes(cache, true, true, true);
  if (s != BITNEST_OK) return s;
  const int64_t step = type == BITNEST_F16 ? 8 : 4;  // values of 16 bytes
  if (misaligned(k) || misaligned(v) || k_token % step || v_token % step ||
      reinterpret_cast<uintptr_t>(start) % 4 || reinterpret_cast<uintptr_t>(count) % 4 ||
      reinterpret_cast<uintptr_t>(pos) % 4 || reinterpret_cast<uintptr_t>(phase) % 8)
    return BITNEST_ERR_MISALIGNED;
  AppendArgs a{k, v, type, k_token, v_token, start, count, pos, phase, magnitude, B, L, Hkv, cap,
               rot, layout == BITNEST_ROPE_PAIRS, planes(cache)};
  return cuda_status(launch_kv_append(a, (cudaStream_t)stream));
}

int bitnest_kv_read(int mode, const bitnest_kv_cache *cache, int64_t B, int64_t cap, int64_t Hkv,
                    const int32_t *start, int64_t L, uint16_t *k, uint16_t *v, void *stream) {
  if (mode != BITNEST_DRAFT && mode != BITNEST_TARGET) return BITNEST_ERR_INVALID_ARG;
  if (!cache_shape_ok(B, cap, Hkv) || L < 0 || L > kMost || (B > 0 && L > kMost / B) ||
      B * L > ((int64_t)1 << 34) / Hkv)
    return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (B == 0 || L == 0) return BITNEST_OK;
  if (!k || !v) return BITNEST_ERR_INVALID_ARG;
  if (cap > 0) {
    const int s = check_planes(cache, true, true, mode == BITNEST_TARGET);
    if (s != BITNEST_OK) return s;
  }
  if (misaligned(k) || misaligned(v) || reinterpret_cast<uintptr_t>(start) % 4)
    return BITNEST_ERR_MISALIGNED;
  ReadArgs a{mode, start, B, L, Hkv, cap, planes(cache), k, v};
  return cuda_status(launch_kv_read(a, (cudaStream_t)stream));
}

int64_t bitnest_prefix_attention_ws_bytes(int64_t B, int64_t L, int64_t H, int64_t Hkv, int64_t P,
                                          int64_t cap) {
  if (!prefix_attention_supported(B, L, H, Hkv, P, cap)) return -BITNEST_ERR_UNSUPPORTED_SHAPE;
  return prefix_attention_ws_bytes(B, L, H, Hkv, P, cap);
}

int bitnest_prefix_attention(int mode, const uint16_t *q, int64_t B, int64_t L, int64_t H,
                             int64_t Hkv, int64_t D, const bitnest_kv_cache *prefix, int64_t P,
                             const bitnest_kv_cache *own, int64_t cap, const int32_t *len,
                             uint16_t *out, float *lse, void *ws, int64_t ws_bytes, void *stream) {
  if (mode != BITNEST_DRAFT && mode != BITNEST_TARGET) return BITNEST_ERR_INVALID_ARG;
  if (D != 128 || !prefix_attention_supported(B, L, H, Hkv, P, cap))
    return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return BITNEST_OK;
  const bool lo = mode == BITNEST_TARGET;
  if (!q || !out || !len) return BITNEST_ERR_INVALID_ARG;
  if (P > 0) {
    const int s = check_planes(prefix, true, true, lo);
    if (s != BITNEST_OK) return s;
  }
  if (cap > 0) {
    const int s = check_planes(own, true, true, lo);
    if (s != BITNEST_OK) return s;
  }
  const int64_t need = prefix_attention_ws_bytes(B, L, H, Hkv, P, cap);
  if (need > 0 && (!ws || ws_bytes < need)) return BITNEST_ERR_INVALID_ARG;
  if (misaligned(q) || misaligned(out) || (need > 0 && misaligned(ws)) ||
      reinterpret_cast<uintptr_t>(len) % 4 || reinterpret_cast<uintptr_t>(lse) % 4)
    return BITNEST_ERR_MISALIGNED;
  PrefixAttnArgs a{mode, q, B, L, H, Hkv, P, cap, planes(prefix, lo), planes(own, lo), len, out, lse, ws};
  return cuda_status(launch_prefix_attention(a, (cudaStream_t)stream));
}

int bitnest_kv_weights(int mode, const uint16_t *q, const float *lse, int64_t B, int64_t L,
                       int64_t H, int64_t Hkv, int64_t D, const uint8_t *k_hi, const uint8_t *k_lo,
                       const uint16_t *k_scale, int64_t cap, const int32_t *len, float *acc,
                       void *stream) {
  if (mode != BITNEST_DRAFT && mode != BITNEST_TARGET) return BITNEST_ERR_INVALID_ARG;
  if (D != 128 || L < 1 || !heads_ok(H, Hkv) || !cache_shape_ok(B, cap, Hkv) || L > kMost ||
      (B > 0 && B * L > kMost / H) || (len && B * Hkv > 65535) ||
      (!len && Hkv * ((cap + 127) / 128) > 0x3fffffff))  // token tiles, counted in 32 bits
    return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (B == 0 || cap == 0) return BITNEST_OK;
  const bool lo = mode == BITNEST_TARGET;
  if (!q || !lse || !k_hi || (lo && !k_lo) || !k_scale || !acc) return BITNEST_ERR_INVALID_ARG;
  if (misaligned(q) || misaligned(k_hi) || (lo && misaligned(k_lo)) || misaligned(k_scale) ||
      reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(acc) % 4 ||
      reinterpret_cast<uintptr_t>(len) % 4)
    return BITNEST_ERR_MISALIGNED;
  KvWeightsArgs a{mode, q, lse, B, L, H, Hkv, cap, k_hi, lo ? k_lo : nullptr, k_scale, len, acc};
  return cuda_status(launch_kv_weights(a, (cudaStream_t)stream));
}

int bitnest_kv_evict(const float *acc, const int32_t *len, int64_t B, int64_t Hkv, int64_t cap,
                     int64_t keep, int64_t sinks, int64_t recent, const bitnest_kv_cache *src,
                     const bitnest_kv_cache *dst, int64_t dst_cap, float *dst_acc, int32_t *kept,
                     int32_t *dst_len, void *stream) {
  if (!cache_shape_ok(B, cap, Hkv) || !cache_shape_ok(B, dst_cap, Hkv))
    return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (keep < 1 || keep > dst_cap || sinks < 0 || recent < 0 || sinks > keep || recent > keep - sinks)
    return BITNEST_ERR_INVALID_ARG;
  if (B * Hkv > 0x7fffffff || (B > 0 && B * Hkv > ((int64_t)1 << 34) / keep))
    return BITNEST_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return BITNEST_OK;
  if (!len || !dst_acc || !kept || !dst_len) return BITNEST_ERR_INVALID_ARG;
  int s = check_planes(dst, true, true, true);
  if (s != BITNEST_OK) return s;
  if (cap > 0) {
    if (!acc) return BITNEST_ERR_INVALID_ARG;
    s = check_planes(src, true, true, true);
    if (s != BITNEST_OK) return s;
    // rows move between CTAs in no order: the new cache is another one
    if (src->k_hi == dst->k_hi || src->k_lo == dst->k_lo || src->k_scale == dst->k_scale ||
        src->v_hi == dst->v_hi || src->v_lo == dst->v_lo || src->v_scale == dst->v_scale ||
        acc == dst_acc || len == dst_len)
      return BITNEST_ERR_INVALID_ARG;
  }
  if (reinterpret_cast<uintptr_t>(acc) % 4 || reinterpret_cast<uintptr_t>(dst_acc) % 4 ||
      reinterpret_cast<uintptr_t>(len) % 4 || reinterpret_cast<uintptr_t>(kept) % 4 ||
      reinterpret_cast<uintptr_t>(dst_len) % 4)
    return BITNEST_ERR_MISALIGNED;
  KvEvictArgs a{acc, len, B, Hkv, cap, dst_cap, keep, sinks, recent, planes(src), planes(dst),
                dst_acc, kept, dst_len};
  return cuda_status(launch_kv_evict(a, (cudaStream_t)stream));
}

}  // extern "C"
