// kvcache.h -- the paged cache as kernels see it, the launchers of
// kvcache.cu and attention.cu, and the E4M3 row format's device helpers.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mfd.h"

namespace mfd {

// mfd_kv_cache with its page size as a shift.
struct CacheView {
  void *k, *v;
  uint8_t *k_exp, *v_exp;
  const int32_t *table;
  int dtype, n_pages, ps_shift, max_pages, Hk, D;
  int64_t page_stride, head_stride, token_stride;  // elements
};

// kvcache.cu
struct AppendLaunch {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  int dtype;                             // MFD_BF16 or MFD_FP16
  int n_req, N, Hq, Hk, D;
  const void *q_w, *k_w;
  float eps;
  const uint64_t *phase;
  int rot_dim, interleaved;
  const int32_t *pos, *ctx_len, *n_nodes;
  void *q_out, *k_out;  // k_out: the keys as a tensor, without a cache
  const CacheView *cache;
  int32_t *status;
};
cudaError_t launch_kv_append(const AppendLaunch &A, cudaStream_t stream);

struct KvReadLaunch {
  CacheView cache;
  int n_req, L_max, dtype;
  const int32_t *start, *length;
  void *k_out, *v_out;
  int32_t *status;
};
cudaError_t launch_kv_read(const KvReadLaunch &A, cudaStream_t stream);

struct KvCommitLaunch {
  CacheView cache;
  int n_req, L;
  const int32_t *ctx_len, *accept_len, *path, *n_nodes;
  int32_t *new_len, *status;
};
cudaError_t launch_kv_commit(const KvCommitLaunch &A, cudaStream_t stream);

// attention.cu
constexpr float ATTENTION_LOG2E = 1.4426950408889634f;
constexpr int ATTENTION_MAX_CTAS = 152;  // GB300's SMs: scratch is sized without asking the device
size_t attention_part_bytes(int M, int D);
int attention_box_rows(int page_size);  // positions of a tensor map's box
struct AttentionLaunch {
  const void *q;
  int64_t q_stride;
  int dtype, n_req, N, Hq;
  CacheView cache;
  const int32_t *ctx_len, *n_nodes;
  const uint32_t *mask;
  float scale;
  void *out;
  float *lse;
  int32_t *status;
  const CUtensorMap *map_k, *map_v;
  int n_sm;
  void *ws;
};
cudaError_t launch_tree_attention(const AttentionLaunch &A, cudaStream_t stream);

#ifdef __CUDACC__
// ---------------------------------------------------------------- elements
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&r);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&r);
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<T>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// ---------------------------------------------------------------- E4M3 rows
constexpr int EXP_NAN = 255;  // the row holds a NaN or an infinity

// The row's byte from the bits of max|x| (NaN orders above infinity, which
// orders above every number, so an integer maximum finds them).  448 * 2^e =
// 1.75 * 2^(e + 8): with max|x| = 1.m * 2^(E - 127), e = E - 135 when 1.m <=
// 1.75 and one more otherwise.
__device__ __forceinline__ int e4m3_code(uint32_t amax_bits) {
  const int E = (int)(amax_bits >> 23);
  if (E == 255) return EXP_NAN;
  const int code = E - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return code < 0 ? 0 : code;
}
// 2^-e of a number's code (0..247): exact, a normal float
__device__ __forceinline__ float e4m3_inv(int code) { return __uint_as_float((uint32_t)(254 - code) << 23); }
// 2^e, subnormal for code 0
__device__ __forceinline__ float e4m3_scale(int code) {
  return code == EXP_NAN ? __int_as_float(0x7FFFFFFF) : __uint_as_float(code ? (uint32_t)code << 23 : 0x400000u);
}
// Largest magnitude to round.  Values come in fp32 (keys after their norm and
// rotation), and what is held must not pass the type's largest.  bf16: only in
// its top binade, code 247, where values in (248, 255.9] * 2^e would round to
// 256 * 2^e.  fp16: the grid's largest number inside is 1.875 * 2^15 = 61440
// from code 135 on; in units of 2^e that is 240, 120, .. -- numbers of the
// grid, a normal one as far as keys go (a norm's row is at most 16 times a
// weight of 65504, a rotation adds sqrt 2: code 139; below 149 it is normal).
template <typename T>
__device__ __forceinline__ float e4m3_limit(int code);
template <>
__device__ __forceinline__ float e4m3_limit<__nv_bfloat16>(int code) { return code >= 247 ? 240.f : 448.f; }
template <>
__device__ __forceinline__ float e4m3_limit<__half>(int code) { return code >= 135 ? 61440.f * e4m3_inv(code) : 448.f; }

// Four floats to four E4M3 bytes, round to nearest even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// Two E4M3 bytes to two floats (exact).
__device__ __forceinline__ float2 e4m3x2_float(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
#endif  // __CUDACC__

}  // namespace mfd
