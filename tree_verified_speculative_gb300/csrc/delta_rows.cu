// delta_rows.cu -- the gated delta rule row after row: few rows, and accepted paths
// (the target's recurrent layers; the method's pages name hybrid targets: model
// card "MFD drafter for Qwen3.5-4B").
//
//   S' = e^g S,  u = beta (v - S'^T k),  S = S' + k u^T,  o = scale S^T q
//
// A warp has 16 columns of one head's state in registers: 4 lanes a float4 of
// each, 8 groups of lanes Dk / 8 rows each.  With both sums of a row made from
// the state before it, kS = S^T k and qS = S^T q,
//
//   u = beta (v - e^g kS),  o = scale (e^g qS + (q . k) u),
//
// three exchanges between the groups serve a row, and warps do not wait for each
// other: a block's warps share the rows' vectors, BATCH of them at a time.  (With
// the groups in different warps and a barrier for each row, 32 accepted paths took
// 48 us.)
#include "delta.h"
#include "kvcache.h"
#include "mfd_device.cuh"

namespace mfd {
namespace {

constexpr int COLS = 16;     // of a warp
constexpr int BATCH = 17;    // rows whose vectors are in shared memory at once: all of a path
constexpr int MAX_DK = 128;
constexpr int PER = MAX_DK / 8;  // rows of the state a lane holds

enum { RULE = 0, COMMIT = 1 };

__device__ __forceinline__ float4 fma4(float a, float4 b, float4 c) {
  return make_float4(fmaf(a, b.x, c.x), fmaf(a, b.y, c.y), fmaf(a, b.z, c.z), fmaf(a, b.w, c.w));
}
// The sum over the eight groups of lanes.
__device__ __forceinline__ float4 group_sum(float4 v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
  }
  return v;
}

template <typename T, int WARPS, int MODE>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) delta_rows_kernel(const DeltaArgs p, int slices) {
  constexpr int W = WARPS * COLS;
  __shared__ float4 k_s[BATCH][MAX_DK / 4], q_s[MODE == COMMIT ? 1 : BATCH][MAX_DK / 4];
  __shared__ uint4 v_s[BATCH][W / 8];
  __shared__ float decay_s[BATCH], beta_s[BATCH], qk_s[BATCH];
  __shared__ int row_s[BATCH], bad_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slice = blockIdx.x % slices, h = blockIdx.x / slices % p.Hv, r = blockIdx.x / slices / p.Hv;
  const int group = lane >> 2, col = slice * W + warp * COLS + (lane & 3) * 4;
  const bool have = col < p.Dv;
  const int hk = h / (p.Hv / p.Hk), per = p.Dk / 8;  // rows of a group: even
  pdl_launch_dependents();
  pdl_wait();

  // lengths and slots; a request whose numbers are wrong has no rows and keeps no state
  int nn = p.n_nodes ? __ldg(p.n_nodes + r) : p.N;
  const int src = p.src ? __ldg(p.src + r) : r;
  const int dst = p.dst ? __ldg(p.dst + r) : src;
  bool ok = nn >= 0 && nn <= p.N && src >= -1 && src < p.n_slots && dst >= -1 && dst < p.n_slots;
  float4 S[PER];
  {
    const float *from = p.s + (((int64_t)src * p.Hv + h) * p.Dk + group * per) * p.Dv + col;
#pragma unroll
    for (int t = 0; t < PER; ++t)
      S[t] = ok && src >= 0 && have && t < per ? *reinterpret_cast<const float4 *>(from + (int64_t)t * p.Dv) : make_float4(0, 0, 0, 0);
  }
  if (per < PER) {  // narrower keys leave elements between the groups': zeros, like the state's rows there
    for (int i = tid; i < BATCH * MAX_DK; i += WARPS * 32) reinterpret_cast<float *>(k_s)[i] = 0.f;
    for (int i = tid; i < (MODE == COMMIT ? 1 : BATCH) * MAX_DK; i += WARPS * 32) reinterpret_cast<float *>(q_s)[i] = 0.f;
    block_sync();
  }
  const int64_t tok0 = (int64_t)r * p.N;
  int rows = nn;
  if (MODE == COMMIT) {
    if (tid == 0) bad_s = 0;
    block_sync();
    rows = ok ? __ldg(p.accept_len + r) + 1 : 0;
    if (rows < 1 || rows > p.L + 1) ok = false;
    const int32_t *path = p.path + (int64_t)r * (p.L + 1);
    if (ok && tid < rows) {
      const int node = __ldg(path + tid);
      const bool good = node < nn && (tid == 0 ? node == 0 : node > __ldg(path + tid - 1));
      if (!good) bad_s = 1;
      row_s[tid] = node;
    }
    block_sync();
    if (bad_s) ok = false;
  }
  if (!ok) {
    if (tid == 0) report(p.status, MFD_ERR_INPUT);
    rows = nn = 0;
  }
  // rows that are not live
  if (MODE == RULE && have)
    for (int i = nn + group; i < p.N; i += 8)
      *reinterpret_cast<uint2 *>(p.out + ((tok0 + i) * p.Hv + h) * p.Dv + col) = make_uint2(0, 0);
  if (!ok) return;

  // The state is S times `kept`, the product of the decays since it was last multiplied
  // out: a row then costs two products an element, not three.
  float kept = 1.f;
  for (int first = 0; first < rows; first += BATCH) {
    const int n = min(BATCH, rows - first);
    if (first) block_sync();
    for (int i = tid; i < n * (W / 8); i += WARPS * 32) {
      const int row = i / (W / 8), c = i % (W / 8), at = slice * W + c * 8;
      const int64_t tok = tok0 + (MODE == COMMIT ? row_s[row] : first + row);
      if (at < p.Dv) v_s[row][c] = __ldg(reinterpret_cast<const uint4 *>(p.v + tok * p.v_stride + h * p.Dv + at));
    }
    // half a warp for a key, half for a query
    for (int i = warp; i < n; i += WARPS) {
      const int64_t tok = tok0 + (MODE == COMMIT ? row_s[i] : first + i);
      const int c = lane & 15;
      const bool is_q = lane >= 16;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (c * 8 < p.Dk && (!is_q || MODE != COMMIT))
        raw = __ldg(reinterpret_cast<const uint4 *>((is_q ? p.q + tok * p.q_stride : p.k + tok * p.k_stride) + hk * p.Dk + c * 8));
      const float g = __ldg(p.g + tok * p.Hv + h), b = __ldg(p.beta + tok * p.Hv + h);
      float x[8], ss = 0.f, qk = 0.f;
      unpack8<T>(raw, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (p.normalize) {
        const float f = rsqrtf(ss + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= f;
      }
      if (MODE != COMMIT) {
#pragma unroll
        for (int e = 0; e < 8; ++e) qk = fmaf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 16), qk);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) qk += __shfl_xor_sync(0xffffffffu, qk, o);
      }
      if (!is_q || MODE != COMMIT) {
        // element e of the vector is element e % per of group e / per; rows of groups are
        // PER floats apart in shared memory, whatever Dk is
        float *to = reinterpret_cast<float *>(is_q ? q_s[i] : k_s[i]);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int at = c * 8 + e;
          if (at < p.Dk) *reinterpret_cast<float2 *>(to + at / per * PER + at % per) = make_float2(x[e], x[e + 1]);
        }
      }
      if (lane == 0) {
        decay_s[i] = expf(g);
        beta_s[i] = b;
        qk_s[i] = qk;
      }
    }
    block_sync();
    for (int i = 0; i < n; ++i) {
      const uint2 raw = reinterpret_cast<const uint2 *>(v_s[i])[warp * (COLS / 4) + (lane & 3)];
      const float2 v0 = unpack2<T>(raw.x), v1 = unpack2<T>(raw.y);
      const float4 v = make_float4(v0.x, v0.y, v1.x, v1.y);
      float4 a = make_float4(0, 0, 0, 0), b = a;
      const float4 *kv = k_s[i] + group * (PER / 4), *qv = q_s[MODE == COMMIT ? 0 : i] + group * (PER / 4);
#pragma unroll
      for (int t = 0; t < PER; t += 4) {
        const float4 k = kv[t / 4];
        a = fma4(k.x, S[t], a);
        a = fma4(k.y, S[t + 1], a);
        a = fma4(k.z, S[t + 2], a);
        a = fma4(k.w, S[t + 3], a);
        if (MODE != COMMIT) {
          const float4 q = qv[t / 4];
          b = fma4(q.x, S[t], b);
          b = fma4(q.y, S[t + 1], b);
          b = fma4(q.z, S[t + 2], b);
          b = fma4(q.w, S[t + 3], b);
        }
      }
      a = group_sum(a);
      if (MODE != COMMIT) b = group_sum(b);
      const float d = decay_s[i] * kept, beta = beta_s[i];
      const float4 u = make_float4(beta * fmaf(-d, a.x, v.x), beta * fmaf(-d, a.y, v.y), beta * fmaf(-d, a.z, v.z),
                                   beta * fmaf(-d, a.w, v.w));
      kept = d;
      if (!(d > 0x1p-40f && d < 0x1p40f)) {  // too small to divide by, or NaN
#pragma unroll
        for (int t = 0; t < PER; ++t) S[t] = make_float4(d * S[t].x, d * S[t].y, d * S[t].z, d * S[t].w);
        kept = 1.f;
      }
      const float up = 1.f / kept;
      const float4 w = make_float4(u.x * up, u.y * up, u.z * up, u.w * up);
#pragma unroll
      for (int t = 0; t < PER; t += 4) {
        const float4 k = kv[t / 4];
        S[t] = fma4(k.x, w, S[t]);
        S[t + 1] = fma4(k.y, w, S[t + 1]);
        S[t + 2] = fma4(k.z, w, S[t + 2]);
        S[t + 3] = fma4(k.w, w, S[t + 3]);
      }
      if (MODE != COMMIT && group == 0 && have) {
        const float qk = qk_s[i];
        *reinterpret_cast<uint2 *>(p.out + ((tok0 + first + i) * p.Hv + h) * p.Dv + col) =
            make_uint2(pack2<T>(p.scale * fmaf(qk, u.x, d * b.x), p.scale * fmaf(qk, u.y, d * b.y)),
                       pack2<T>(p.scale * fmaf(qk, u.z, d * b.z), p.scale * fmaf(qk, u.w, d * b.w)));
      }
    }
  }
  if (dst >= 0 && have) {
    float *to = p.s + (((int64_t)dst * p.Hv + h) * p.Dk + group * per) * p.Dv + col;
#pragma unroll
    for (int t = 0; t < PER; ++t)
      if (t < per)
        *reinterpret_cast<float4 *>(to + (int64_t)t * p.Dv) = make_float4(kept * S[t].x, kept * S[t].y, kept * S[t].z, kept * S[t].w);
  }
}

template <typename T, int WARPS, int MODE>
cudaError_t launch_width(const DeltaArgs &A, cudaStream_t stream) {
  const int slices = (A.Dv + WARPS * COLS - 1) / (WARPS * COLS);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)A.n_req * A.Hv * slices));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = stream;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, delta_rows_kernel<T, WARPS, MODE>, A, slices);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int MODE>
cudaError_t launch_mode(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  // narrower slices where heads alone leave SMs without work
  const int64_t heads = (int64_t)A.n_req * A.Hv;
  if (heads * ((A.Dv + 63) / 64) <= n_sm) return launch_width<T, 2, MODE>(A, stream);
  return launch_width<T, 4, MODE>(A, stream);
}
template <int MODE>
cudaError_t launch_type(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  return A.dtype == MFD_BF16 ? launch_mode<__nv_bfloat16, MODE>(A, n_sm, stream) : launch_mode<__half, MODE>(A, n_sm, stream);
}

}  // namespace

cudaError_t launch_delta_rows(const DeltaArgs &A, int n_sm, cudaStream_t stream) { return launch_type<RULE>(A, n_sm, stream); }
cudaError_t launch_delta_commit(const DeltaArgs &A, int n_sm, cudaStream_t stream) { return launch_type<COMMIT>(A, n_sm, stream); }

}  // namespace mfd
