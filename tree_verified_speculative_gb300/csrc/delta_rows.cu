// delta_rows.cu -- the gated delta rule row after row: few rows, and accepted paths
// (the target's recurrent layers; the method's pages name hybrid targets: model
// card "MFD drafter for Qwen3.5-4B").
//
//   S' = e^g S,  u = beta (v - S'^T k),  S = S' + k u^T,  o = scale S^T q
//
// A block holds W columns of one head's state in registers, a thread a float4
// of Dk / RG rows (RG groups of threads share the columns).  With both sums of
// a row made from the state before it, kS = S^T k and qS = S^T q,
//
//   u = beta (v - e^g kS),  o = scale (e^g qS + (q . k) u),
//
// one exchange between the groups serves a row, and a row's dot product q . k
// does not wait for the state.
#include "delta.h"
#include "kvcache.h"
#include "mfd_device.cuh"

namespace mfd {
namespace {

constexpr int THREADS = 256;
constexpr int BATCH = 16;    // rows whose vectors are in shared memory at once
constexpr int MAX_DK = 128;

enum { RULE = 0, COMMIT = 1 };

__device__ __forceinline__ float4 fma4(float a, float4 b, float4 c) {
  return make_float4(fmaf(a, b.x, c.x), fmaf(a, b.y, c.y), fmaf(a, b.z, c.z), fmaf(a, b.w, c.w));
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
__device__ __forceinline__ float4 shfl4(float4 v, int o) {
  return make_float4(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o),
                     __shfl_xor_sync(0xffffffffu, v.z, o), __shfl_xor_sync(0xffffffffu, v.w, o));
}

template <typename T, int W, int MODE>
__global__ void __launch_bounds__(THREADS) delta_rows_kernel(const DeltaArgs p, int slices) {
  constexpr int LW = W / 4, RG = THREADS / LW;      // lanes of a row, groups
  constexpr int PER = MAX_DK / RG;                  // rows of the state a thread holds
  constexpr int WARPS = THREADS / 32;
  __shared__ float k_s[BATCH][MAX_DK], q_s[BATCH][MAX_DK];
  __shared__ float4 v_s[BATCH][LW];
  __shared__ float decay_s[BATCH], beta_s[BATCH], qk_s[BATCH];
  __shared__ float4 sum_s[2][2][WARPS][LW];  // [row mod 2][keys, queries][warp][lane]
  __shared__ int row_s[DELTA_MAX_DEPTH + 1], bad_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slice = blockIdx.x % slices, h = blockIdx.x / slices % p.Hv, r = blockIdx.x / slices / p.Hv;
  const int col = slice * W + (tid % LW) * 4, rg = tid / LW;
  const bool have = col < p.Dv;
  const int hk = h / (p.Hv / p.Hk);
  pdl_launch_dependents();
  pdl_wait();

  // lengths and slots; a request whose numbers are wrong has no rows and keeps no state
  int nn = p.n_nodes ? __ldg(p.n_nodes + r) : p.N;
  const int src = p.src ? __ldg(p.src + r) : r;
  const int dst = p.dst ? __ldg(p.dst + r) : src;
  bool ok = nn >= 0 && nn <= p.N && src >= -1 && src < p.n_slots && dst >= -1 && dst < p.n_slots;
  const int64_t tok0 = (int64_t)r * p.N;
  if (tid == 0) bad_s = 0;
  block_sync();
  int rows = nn;
  if (MODE == COMMIT) {
    rows = ok ? __ldg(p.accept_len + r) + 1 : 0;
    if (rows < 1 || rows > p.L + 1) ok = false;
    const int32_t *path = p.path + (int64_t)r * (p.L + 1);
    if (ok && tid < rows) {
      const int node = __ldg(path + tid);
      const bool good = node < nn && (tid == 0 ? node == 0 : node > __ldg(path + tid - 1));
      if (!good) bad_s = 1;
      row_s[tid] = node;
    }
  }
  block_sync();
  if (bad_s) ok = false;
  if (!ok) {
    if (tid == 0) report(p.status, MFD_ERR_INPUT);
    rows = 0;
    nn = 0;
  }
  // rows that are not live
  if (MODE != COMMIT && have)
    for (int i = nn + rg; i < p.N; i += RG)
      *reinterpret_cast<uint2 *>(p.out + ((tok0 + i) * p.Hv + h) * p.Dv + col) = make_uint2(0, 0);
  if (!ok) return;

  float4 S[PER];
  const float *from = p.s + ((int64_t)src * p.Hv + h) * p.Dk * p.Dv + col;
#pragma unroll
  for (int t = 0; t < PER; ++t) {
    const int row = rg + RG * t;
    S[t] = src >= 0 && have && row < p.Dk ? *reinterpret_cast<const float4 *>(from + (int64_t)row * p.Dv) : make_float4(0, 0, 0, 0);
  }
  // vectors of rows at(first) .. at(first + n - 1): half a warp for a key, half for a query
  auto load_rows = [&](int first, int n, auto at) {
    for (int i = warp; i < n; i += WARPS) {
      const int64_t tok = tok0 + at(first + i);
      const int c = lane & 15;
      const bool is_q = lane >= 16;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (c * 8 < p.Dk && (!is_q || MODE != COMMIT))
        raw = *reinterpret_cast<const uint4 *>(is_q ? p.q + tok * p.q_stride + hk * p.Dk + c * 8
                                                    : p.k + tok * p.k_stride + hk * p.Dk + c * 8);
      uint2 vr = make_uint2(0, 0);
      if (lane < LW && slice * W + lane * 4 < p.Dv)
        vr = *reinterpret_cast<const uint2 *>(p.v + tok * p.v_stride + h * p.Dv + slice * W + lane * 4);
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
#pragma unroll
      for (int e = 0; e < 8; ++e) qk = fmaf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 16), qk);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) qk += __shfl_xor_sync(0xffffffffu, qk, o);
      float *to = (is_q ? q_s[i] : k_s[i]) + c * 8;
      *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4 *>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
      if (lane < LW) {
        const float2 a = unpack2<T>(vr.x), d = unpack2<T>(vr.y);
        v_s[i][lane] = make_float4(a.x, a.y, d.x, d.y);
      }
      if (lane == 0) {
        decay_s[i] = expf(g);
        beta_s[i] = b;
        qk_s[i] = qk;
      }
    }
  };
  uint32_t turn = 0;
  // one row from shared memory; `out`: where this slice's columns of its output go, or NULL
  auto step = [&](int i, uint16_t *out) {
    float4 a = make_float4(0, 0, 0, 0), b = a;
#pragma unroll
    for (int t = 0; t < PER; ++t) {
      a = fma4(k_s[i][rg + RG * t], S[t], a);
      if (MODE != COMMIT) b = fma4(q_s[i][rg + RG * t], S[t], b);
    }
#pragma unroll
    for (int o = LW; o < 32; o <<= 1) {
      a = add4(a, shfl4(a, o));
      if (MODE != COMMIT) b = add4(b, shfl4(b, o));
    }
    float4(*sum)[WARPS][LW] = sum_s[turn & 1];
    ++turn;
    if (lane < LW) {
      sum[0][warp][lane] = a;
      if (MODE != COMMIT) sum[1][warp][lane] = b;
    }
    block_sync();
    a = b = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      a = add4(a, sum[0][w][tid % LW]);
      if (MODE != COMMIT) b = add4(b, sum[1][w][tid % LW]);
    }
    const float d = decay_s[i], beta = beta_s[i], qk = qk_s[i];
    const float4 v = v_s[i][tid % LW];
    const float4 u = make_float4(beta * fmaf(-d, a.x, v.x), beta * fmaf(-d, a.y, v.y), beta * fmaf(-d, a.z, v.z),
                                 beta * fmaf(-d, a.w, v.w));
#pragma unroll
    for (int t = 0; t < PER; ++t) {
      const float k = k_s[i][rg + RG * t];
      S[t] = make_float4(fmaf(k, u.x, d * S[t].x), fmaf(k, u.y, d * S[t].y), fmaf(k, u.z, d * S[t].z), fmaf(k, u.w, d * S[t].w));
    }
    if (out && rg == 0 && have)
      *reinterpret_cast<uint2 *>(out) =
          make_uint2(pack2<T>(p.scale * fmaf(qk, u.x, d * b.x), p.scale * fmaf(qk, u.y, d * b.y)),
                     pack2<T>(p.scale * fmaf(qk, u.z, d * b.z), p.scale * fmaf(qk, u.w, d * b.w)));
  };
  auto out_of = [&](int i) { return p.out + ((tok0 + i) * p.Hv + h) * p.Dv + col; };

  for (int first = 0; first < rows; first += BATCH) {
    const int n = min(BATCH, rows - first);
    if (first) block_sync();
    load_rows(first, n, [&](int j) { return MODE == COMMIT ? row_s[j] : j; });
    block_sync();
    for (int i = 0; i < n; ++i) step(i, MODE == COMMIT ? nullptr : out_of(first + i));
  }
  if (dst >= 0 && have) {
    float *to = p.s + ((int64_t)dst * p.Hv + h) * p.Dk * p.Dv + col;
#pragma unroll
    for (int t = 0; t < PER; ++t) {
      const int row = rg + RG * t;
      if (row < p.Dk) *reinterpret_cast<float4 *>(to + (int64_t)row * p.Dv) = S[t];
    }
  }
}

template <typename T, int W, int MODE>
cudaError_t launch_width(const DeltaArgs &A, cudaStream_t stream) {
  const int slices = (A.Dv + W - 1) / W;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)A.n_req * A.Hv * slices));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, delta_rows_kernel<T, W, MODE>, A, slices);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int MODE>
cudaError_t launch_mode(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  // narrower slices where heads alone leave SMs without work
  const int64_t heads = (int64_t)A.n_req * A.Hv;
  if (heads * ((A.Dv + 63) / 64) <= n_sm) return launch_width<T, 32, MODE>(A, stream);
  if (heads * ((A.Dv + 127) / 128) <= n_sm) return launch_width<T, 64, MODE>(A, stream);
  return launch_width<T, 128, MODE>(A, stream);
}
template <int MODE>
cudaError_t launch_type(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  return A.dtype == MFD_BF16 ? launch_mode<__nv_bfloat16, MODE>(A, n_sm, stream) : launch_mode<__half, MODE>(A, n_sm, stream);
}

}  // namespace

cudaError_t launch_delta_rows(const DeltaArgs &A, int n_sm, cudaStream_t stream) { return launch_type<RULE>(A, n_sm, stream); }
cudaError_t launch_delta_commit(const DeltaArgs &A, int n_sm, cudaStream_t stream) { return launch_type<COMMIT>(A, n_sm, stream); }

}  // namespace mfd
