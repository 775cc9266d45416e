// attention.cu -- attention of a request's rows (the tree's nodes under the
// tree mask, one token, or a stretch of a prompt) over the paged cache
// (project page "Multi-Future Drafting", How it works, step 3, Figure 2 (c):
// one target pass scores every node of the tree).
//
// The plain form: one block per (request, row, query head).  A warp takes
// every fourth position, its lanes share the head's D elements, and the
// running maximum, sum and weighted values of the four warps are joined at
// the end.  Every row reads its whole context by itself.
#include "kvcache.h"
#include "mfd_device.cuh"

namespace mfd {
namespace {

constexpr int THREADS = 128;
constexpr int WARPS = 4;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// Element e of entry `at` as a float.
template <typename T, bool E4M3>
__device__ __forceinline__ float load_element(const void *base, int64_t at, float s) {
  if (E4M3) return e4m3x2_float(static_cast<const uint8_t *>(base)[at]).x * s;
  const uint16_t w = static_cast<const uint16_t *>(base)[at];
  return unpack2<T>(w).x;
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(THREADS) attention_kernel(const AttentionLaunch A) {
  __shared__ float m_s[WARPS], l_s[WARPS], o_s[WARPS][256];
  const CacheView &cv = A.cache;
  const int D = cv.D, G = A.Hq / cv.Hk;
  const int hq = blockIdx.x, n = blockIdx.y, q = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hd = hq / G;
  int ctx = A.ctx_len[q], nn = A.n_nodes ? A.n_nodes[q] : A.N;
  const int64_t cap = (int64_t)cv.max_pages << cv.ps_shift;
  if (ctx < 0 || nn < 0 || nn > A.N || (int64_t)ctx + nn > cap) {
    if (threadIdx.x == 0) report(A.status, MFD_ERR_INPUT);
    nn = 0;
  }
  const int64_t row = (int64_t)q * A.N + n;
  float qv[8], acc[8];
  const uint16_t *qp = static_cast<const uint16_t *>(A.q) + row * A.q_stride + (int64_t)hq * D;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = lane + 32 * i;
    qv[i] = d < D && n < nn ? unpack2<T>(qp[d]).x * A.scale * LOG2E : 0.f;
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int W32 = (A.N + 31) / 32;
  const int T_end = n < nn ? ctx + nn : 0;
  for (int t = warp; t < T_end; t += WARPS) {
    if (t >= ctx) {
      const int j = t - ctx;
      const bool seen = A.mask ? (A.mask[row * W32 + (j >> 5)] >> (j & 31)) & 1u : j <= n;
      if (!seen) continue;
    }
    const int page = cv.table[(size_t)q * cv.max_pages + (t >> cv.ps_shift)];
    if (page < 0 || page >= cv.n_pages) {
      report(A.status, MFD_ERR_INPUT);
      continue;
    }
    const int slot = t & ((1 << cv.ps_shift) - 1);
    const int64_t at = page * cv.page_stride + hd * cv.head_stride + slot * cv.token_stride;
    const int64_t ex = (((int64_t)page * cv.Hk + hd) << cv.ps_shift) + slot;
    const float ks = E4M3 ? e4m3_scale(cv.k_exp[ex]) : 1.f, vs = E4M3 ? e4m3_scale(cv.v_exp[ex]) : 1.f;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i;
      if (d < D) z = fmaf(qv[i], load_element<T, E4M3>(cv.k, at + d, ks), z);
    }
    z = warp_sum(z);
    const float m2 = fmaxf(m, z);
    const float a = m == -INFINITY ? 0.f : exp2f(m - m2), p = exp2f(z - m2);
    l = l * a + p;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i;
      if (d < D) acc[i] = acc[i] * a + p * load_element<T, E4M3>(cv.v, at + d, vs);
    }
    m = m2;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) o_s[warp][lane + 32 * i] = acc[i];
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  block_sync();
  float mx = -INFINITY, sum = 0.f, w[WARPS];
#pragma unroll
  for (int i = 0; i < WARPS; ++i) mx = fmaxf(mx, m_s[i]);
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    w[i] = m_s[i] == -INFINITY ? 0.f : exp2f(m_s[i] - mx);
    sum += w[i] * l_s[i];
  }
  uint16_t *op = static_cast<uint16_t *>(A.out) + (row * A.Hq + hq) * D;
  for (int d = threadIdx.x; d < D; d += THREADS) {
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) o += w[i] != 0.f ? w[i] * o_s[i][d] : 0.f;
    op[d] = (uint16_t)pack2<T>(l_s[0] == 0.f && sum == 0.f ? 0.f : o / sum, 0.f);
  }
  if (A.lse && threadIdx.x == 0) A.lse[row * A.Hq + hq] = mx == -INFINITY ? -INFINITY : mx * LN2 + logf(sum);
}

}  // namespace

cudaError_t launch_tree_attention(const AttentionLaunch &A, cudaStream_t stream) {
  const dim3 grid(A.Hq, A.N, A.n_req);
  const bool e4m3 = A.cache.dtype == MFD_E4M3;
  if (A.dtype == MFD_BF16) {
    if (e4m3)
      attention_kernel<__nv_bfloat16, true><<<grid, THREADS, 0, stream>>>(A);
    else
      attention_kernel<__nv_bfloat16, false><<<grid, THREADS, 0, stream>>>(A);
  } else {
    if (e4m3)
      attention_kernel<__half, true><<<grid, THREADS, 0, stream>>>(A);
    else
      attention_kernel<__half, false><<<grid, THREADS, 0, stream>>>(A);
  }
  return cudaGetLastError();
}

}  // namespace mfd
