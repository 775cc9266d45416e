// delta_tc.cuh -- what the tensor-core forms of the delta rule share
// (delta_chunk.cu, delta_tree.cu).
#pragma once

#include "delta.h"
#include "kvcache.h"
#include "mfd_device.cuh"
#include "tc16.cuh"

namespace mfd {
namespace {

constexpr float LEAST_LOG = -1e5f;  // of a decay: e^-1e5 is 0 in fp32, and sums of it stay finite

__device__ __forceinline__ float max_nan(float a, float b, float c) {  // largest magnitude; NaN if there is one
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return y;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }
// 2^n and its inverse so that m * 2^n has exponent `to`: from m's bits, both normal.
__device__ __forceinline__ float power_for(float m, int to, float &inverse) {
  int b = 254 + to - (int)(__float_as_uint(m) >> 23);
  b = max(1, min(253, b));
  inverse = __uint_as_float((uint32_t)(254 - b) << 23);
  return __uint_as_float((uint32_t)b << 23);
}
// Two numbers as halves: hi + lo.
__device__ __forceinline__ void halves(float a, float b, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}
// A number as the sum of two floats.
struct Two {
  float hi, lo;
};
constexpr float LOG2E_HI = 0x1.715476p+0f, LOG2E_LO = 0x1.4ae0cp-26f;  // log2 e
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), x = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, x)), __fsub_rn(b, x))};
}
__device__ __forceinline__ Two two_sum(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  const float lo = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)), hi = __fadd_rn(s.hi, lo);
  return {hi, __fsub_rn(lo, __fsub_rn(hi, s.hi))};
}
__device__ __forceinline__ Two two_product(float a, float hi, float lo) {
  const float p = __fmul_rn(a, hi);
  return {p, __fmaf_rn(a, lo, __fmaf_rn(a, hi, -p))};
}
template <typename T>
__device__ __forceinline__ float to_float(uint16_t x) { return unpack2<T>(x).x; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// Lengths and slots of request r.
struct Request {
  int nn, src, dst;
  bool ok;
};
__device__ __forceinline__ Request request(const DeltaArgs &p, int r) {
  Request q;
  q.nn = p.n_nodes ? __ldg(p.n_nodes + r) : p.N;
  q.src = p.src ? __ldg(p.src + r) : r;
  q.dst = p.dst ? __ldg(p.dst + r) : q.src;
  q.ok = q.nn >= 0 && q.nn <= p.N && q.src >= -1 && q.src < p.n_slots && q.dst >= -1 && q.dst < p.n_slots;
  return q;
}

}  // namespace
}  // namespace mfd
