// Internal launchers (C++), called only by the C ABI in capi.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace bitnest {

struct LinearArgs {
  int mode;               // 0 draft, 1 target
  const uint8_t *hi;      // [N, K/2]
  const uint8_t *lo;      // [N, K/2] (target)
  const uint16_t *scale;  // fp16 [N, K/128]
  const int8_t *xq;       // [M, K]
  const float *xscale;    // [M] or [M, K/128]
  const int32_t *xsum;    // [M, K/128] or null (the kernels form the sums)
  const uint16_t *bias;   // fp16 [N] or null
  float *y;               // [M, N]
  int32_t *S;             // debug group sums [M, N, K/128] (null unless debug)
  int64_t M, N, K;
  int act_group;          // 0 or 128
  bool overlap;           // launch with programmatic dependent launch
  // scratch of the tensor-core path's split K (null: no split), its bytes;
  // its counter area is zero before the call and zero again after it
  void *ws = nullptr;
  int64_t ws_bytes = 0;
};

cudaError_t launch_pack(const uint8_t *uh, const uint8_t *ul, int64_t N, int64_t K, uint8_t *hi,
                        uint8_t *lo, cudaStream_t st);
cudaError_t launch_pack_weights(const uint16_t *w, int64_t N, int64_t K, uint8_t *hi,
                                uint8_t *lo, uint16_t *scale, cudaStream_t st);
cudaError_t launch_quantize(const uint16_t *x, int64_t M, int64_t K, int act_group, int8_t *xq,
                            float *xs, int32_t *xsum, cudaStream_t st);
cudaError_t launch_act_group_sums(const int8_t *xq, int64_t M, int64_t K, int32_t *xsum,
                                  cudaStream_t st);
// Decode attention over a nested KV cache (D = 128, H / Hkv in {1,2,4,8}).
bool nested_attention_supported(int64_t H, int64_t Hkv, int64_t D, int64_t T);
cudaError_t launch_nested_attention(int mode, const uint16_t *q, int64_t H, int64_t Hkv,
                                    int64_t T, const uint8_t *k_hi, const uint8_t *k_lo,
                                    const uint16_t *k_scale, const uint8_t *v_hi,
                                    const uint8_t *v_lo, const uint16_t *v_scale, float *out,
                                    cudaStream_t st);
// Hadamard rotation x H / sqrt(K) + per-token quantisation (K = p or 28 p,
// p a power of two, K <= 32768).
bool hadamard_supported(int64_t K);
cudaError_t launch_hadamard_quantize(const uint16_t *x, int64_t M, int64_t K, int8_t *xq,
                                     float *xs, int32_t *xsum, cudaStream_t st);

// Rotary positions (x, y types: 0 fp16, 1 fp32).
struct RopeArgs {
  const void *x;
  int x_type;
  int64_t x_token, x_head;  // strides in elements
  void *y;
  int y_type;
  int64_t y_token, y_head;
  const int32_t *pos;     // [M]
  const uint64_t *phase;  // [rot / 2]
  float mag, sign;
  int64_t M, heads, D, rot;
  bool pairs;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st);

// Six planes of a nested KV cache, rows (b * cap + t) * Hkv + j.
struct KvPlanes {
  uint8_t *k_hi, *k_lo;
  uint16_t *k_scale;
  uint8_t *v_hi, *v_lo;
  uint16_t *v_scale;
};
struct AppendArgs {
  const void *k, *v;  // [B * L, Hkv, 128], token strides in elements
  int type;
  int64_t k_token, v_token;
  const int32_t *start, *count, *pos;
  const uint64_t *phase;  // null: the keys are turned already
  float mag;
  int64_t B, L, Hkv, cap, rot;
  bool pairs;
  KvPlanes cache;
};
cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t st);
struct ReadArgs {
  int mode;
  const int32_t *start;  // null: 0
  int64_t B, L, Hkv, cap;
  KvPlanes cache;
  uint16_t *k, *v;  // fp16 [B, L, Hkv, 128]
};
cudaError_t launch_kv_read(const ReadArgs &a, cudaStream_t st);

// Attention of a batch over one prefix and each sequence's own tokens.
struct PrefixAttnArgs {
  int mode;
  const uint16_t *q;  // fp16 [B, L, H, 128]
  int64_t B, L, H, Hkv, P, cap;
  KvPlanes prefix, own;
  const int32_t *len;  // [B]
  uint16_t *out;       // fp16 [B, L, H, 128]
  float *lse;          // [B, L, H] or null
  void *ws;
};
bool prefix_attention_supported(int64_t B, int64_t L, int64_t H, int64_t Hkv, int64_t P,
                                int64_t cap);
int64_t prefix_attention_ws_bytes(int64_t B, int64_t L, int64_t H, int64_t Hkv, int64_t P,
                                  int64_t cap);
cudaError_t launch_prefix_attention(const PrefixAttnArgs &a, cudaStream_t st);
cudaError_t read_wait_timeout_prefix(int *flag, bool reset);

// Attention weight that each cached token received, added to acc [B, Hkv, cap]
// (len null: acc [Hkv, cap], every query sees every token).
struct KvWeightsArgs {
  int mode;
  const uint16_t *q;
  const float *lse;
  int64_t B, L, H, Hkv, cap;
  const uint8_t *k_hi, *k_lo;
  const uint16_t *k_scale;
  const int32_t *len;
  float *acc;
};
cudaError_t launch_kv_weights(const KvWeightsArgs &a, cudaStream_t st);
namespace evict {
cudaError_t launch_weights_tc(const KvWeightsArgs &a, cudaStream_t st);  // len null
}
cudaError_t read_wait_timeout_weights(int *flag, bool reset);

struct KvEvictArgs {
  const float *acc;  // [B, Hkv, cap]
  const int32_t *len;
  int64_t B, Hkv, cap, cap_out, keep, sinks, recent;
  KvPlanes src, dst;
  float *acc_out;     // [B, Hkv, cap_out]
  int32_t *kept;      // [B, Hkv, keep]
  int32_t *len_out;   // [B]
};
cudaError_t launch_kv_evict(const KvEvictArgs &a, cudaStream_t st);

// Largest M * K the GEMV kernels can stage in shared memory.
bool gemv_fits(int64_t M, int64_t K);
cudaError_t launch_gemv(const LinearArgs &a, cudaStream_t st);

// TMA-ring decode GEMV (K a multiple of 1024).
bool gemv_tma_supported(int64_t M, int64_t N, int64_t K);
cudaError_t launch_gemv_tma(const LinearArgs &a, cudaStream_t st);
cudaError_t read_wait_timeout_gemv(int *flag, bool reset);

// tcgen05 tensor-core GEMM (any M).
bool tc_supported(int64_t M, int64_t N, int64_t K);
cudaError_t launch_tc(const LinearArgs &a, cudaStream_t st);
// Scratch bytes the tensor-core path splits K with for this shape (0: none).
int64_t tc_ws_bytes(int64_t M, int64_t N, int64_t K);
// Size and device address (looked up once per device) of the library's own
// static split-K scratch.
constexpr int64_t kStaticWsBytes = int64_t(12) << 20;
cudaError_t tc_static_ws(void **ws);
// Zero the arrival counters of that scratch (after a bounded wait gave up).
cudaError_t tc_static_ws_clear_counters(cudaStream_t st);

// The flag a bounded wait sets when it gives up (synchronous read).
cudaError_t read_wait_timeout(int *flag, bool reset);
// Test hook: a wait that gives up (sets the flag above).
cudaError_t launch_wait_probe(cudaStream_t st);

}  // namespace bitnest
