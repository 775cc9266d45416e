// norms.cu -- norms with gates around a recurrent layer's output and around a
// block.
//
//   gated     out = x / sqrt(mean x^2 + eps) * w * act(gate), a head's row of D
//             each
//   residual  y' = y, or its norm; r = residual + scale * act(gate) * y';
//             x = r / sqrt(mean r^2 + eps) * w_pre, from the sum before it is
//             rounded
//
// Both move bytes: each element is read once and written once in 16 bytes, sums
// are fp32.
//
// The gated norm of 16,000 tokens of 32 heads of 128 takes 60 us, 6.6 TB/s; the
// residual form of 15,500 rows of 2560 with a gate for each 66 us, 6.0 TB/s.
#include "delta.h"
#include "kvcache.h"
#include "mfd_device.cuh"

namespace mfd {
namespace {

// A sigmoid is 2^-32 / (2^-32 + 2^-32 e^-x): the sum and its inverse stay far inside fp32
// where those of 1 + e^-x do not (below -87, where silu is still a normal bf16 number).  The
// last product may be no normal number; it is then known to 2^-150, next to nothing of a
// 16-bit type's smallest step.
__device__ __forceinline__ float activate(float x, int act) {
  if (act == MFD_ACT_NONE) return x;
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(x, -1.4426950408889634f, -32.f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(0x1p-32f + e));
  s *= 0x1p-32f;
  return act == MFD_ACT_SIGMOID ? s : x * s;          // silu of -inf is NaN, as -inf / (1 + inf) is
}

// ------------------------------------------------------------------ gated

// A row of D elements is LR lanes of 8 (LR: the power of two at or above D / 8);
// a lane has U rows in flight.
constexpr int GATED_THREADS = 256;
template <typename T, int LR, int U>
__global__ void __launch_bounds__(GATED_THREADS) gated_norm_kernel(const GatedNormArgs p) {
  constexpr int PER = GATED_THREADS / LR;  // rows of the block at once
  pdl_launch_dependents();
  pdl_wait();
  const int c = threadIdx.x & (LR - 1);
  const bool in_row = c * 8 < p.D;
  const uint32_t rows = (uint32_t)p.T * p.heads;  // below 2^31
  const uint32_t row0 = blockIdx.x * (PER * U) + threadIdx.x / LR;
  uint4 x[U], z[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t row = row0 + u * PER;
    x[u] = z[u] = make_uint4(0, 0, 0, 0);
    if (in_row && row < rows) {
      const uint32_t t = row / (uint32_t)p.heads, h = row - t * p.heads;
      x[u] = *reinterpret_cast<const uint4 *>(p.x + t * p.x_stride + h * p.D + c * 8);
      z[u] = *reinterpret_cast<const uint4 *>(p.gate + t * p.gate_stride + h * p.D + c * 8);
    }
  }
  float w[8];
  unpack8<T>(in_row ? __ldg(reinterpret_cast<const uint4 *>(p.w) + c) : make_uint4(0, 0, 0, 0), w);
  const float per_d = 1.f / (float)p.D;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t row = row0 + u * PER;
    float a[8], b[8], ss = 0.f;
    unpack8<T>(x[u], a);
    unpack8<T>(z[u], b);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], ss);
#pragma unroll
    for (int o = 1; o < LR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(fmaf(ss, per_d, p.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = a[i] * r * w[i] * activate(b[i], p.act);
    if (in_row && row < rows) *reinterpret_cast<uint4 *>(p.out + (int64_t)row * p.D + c * 8) = pack8<T>(a);
  }
}

template <typename T, int LR>
cudaError_t launch_gated(const GatedNormArgs &A, cudaLaunchConfig_t &cfg) {
  const int64_t rows = (int64_t)A.T * A.heads;
  constexpr int U = 4, PER = GATED_THREADS / LR;
  cfg.blockDim = dim3(GATED_THREADS);
  cfg.gridDim = dim3((unsigned)((rows + PER * U - 1) / (PER * U)));
  return cudaLaunchKernelEx(&cfg, gated_norm_kernel<T, LR, U>, A);
}
template <typename T>
cudaError_t launch_gated_width(const GatedNormArgs &A, cudaLaunchConfig_t &cfg) {
  if (A.D <= 32) return launch_gated<T, 4>(A, cfg);
  if (A.D <= 64) return launch_gated<T, 8>(A, cfg);
  if (A.D <= 128) return launch_gated<T, 16>(A, cfg);
  return launch_gated<T, 32>(A, cfg);
}

// ------------------------------------------------------------------ residual

// The sum of x over the block; `buf` holds a float for every warp and is free
// again after the next barrier.
__device__ __forceinline__ float block_sum(float x, float *buf) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  block_sync();
  const int lane = threadIdx.x & 31, warps = (int)(blockDim.x >> 5);
  return warp_sum(lane < warps ? buf[lane] : 0.f);
}

// A block walks tokens, CH chunks of 8 elements a thread, with the next token's
// loads in flight and the weights in registers.
template <typename T, int CH, int REGS>
__global__ void __maxnreg__(REGS) residual_norm_kernel(const ResidualNormArgs p) {
  __shared__ float sum_s[2][2][16];  // [token mod 2][norm]
  pdl_launch_dependents();
  pdl_wait();
  uint4 y[CH], r[CH], z[CH], wa[CH], wb[CH];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int e = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
      if (e < p.H) {
        y[i] = *reinterpret_cast<const uint4 *>(p.y + t * p.H + e);
        r[i] = *reinterpret_cast<const uint4 *>(p.residual + t * p.H + e);
        if (p.gate) z[i] = *reinterpret_cast<const uint4 *>(p.gate + t * p.gate_stride + e);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int e = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
    y[i] = r[i] = z[i] = wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
    if (e < p.H && p.w_post) wa[i] = __ldg(reinterpret_cast<const uint4 *>(p.w_post + e));
    if (e < p.H && p.w_pre) wb[i] = __ldg(reinterpret_cast<const uint4 *>(p.w_pre + e));
  }
  const float per_h = 1.f / (float)p.H;
  load(blockIdx.x);
  int turn = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
    const int64_t at = t * p.H;
    float norm = 1.f;
    if (p.w_post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float a[8];
        unpack8<T>(y[i], a);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(a[k], a[k], ss);
      }
      norm = rsqrtf(fmaf(block_sum(ss, sum_s[turn][0]), per_h, p.eps));
    }
    float sum[CH][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int e = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
      float a[8], b[8], c[8];
      unpack8<T>(y[i], a);
      unpack8<T>(r[i], b);
      if (p.w_post) {
        unpack8<T>(wa[i], c);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = a[k] * norm * c[k];
      }
      if (p.gate) {
        unpack8<T>(z[i], c);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] *= activate(c[k], p.act);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sum[i][k] = e < p.H ? fmaf(p.scale, a[k], b[k]) : 0.f;
        ss = fmaf(sum[i][k], sum[i][k], ss);
      }
    }
    // The next token's rows: other rows than this token's outputs, also where those go
    // over the inputs.
    if (t + gridDim.x < p.T) load(t + gridDim.x);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int e = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
      if (e < p.H) *reinterpret_cast<uint4 *>(p.residual_out + at + e) = pack8<T>(sum[i]);
    }
    if (!p.w_pre) continue;
    norm = rsqrtf(fmaf(block_sum(ss, sum_s[turn][1]), per_h, p.eps));
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int e = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
      float c[8];
      unpack8<T>(wb[i], c);
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = sum[i][k] * norm * c[k];
      if (e < p.H) *reinterpret_cast<uint4 *>(p.x_out + at + e) = pack8<T>(c);
    }
  }
}

template <typename T, int CH, int REGS>
cudaError_t launch_chunks(const ResidualNormArgs &A, int threads, int n_sm, cudaLaunchConfig_t &cfg) {
  // as many blocks as are resident
  const int fit = 65536 / (threads * REGS), blocks = n_sm * (fit < 1 ? 1 : fit > 32 ? 32 : fit);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.gridDim = dim3((unsigned)(A.T < blocks ? A.T : blocks));
  return cudaLaunchKernelEx(&cfg, residual_norm_kernel<T, CH, REGS>, A);
}
// Two chunks a thread where 512 threads have a row so: a block of few warps waits less
// for its sums, and more blocks are resident (rows of 2560 at 6.1 TB/s, with one chunk a
// thread 5.7; of 4096 5.5 and 5.6).  80 registers a thread, which spill a little, where
// they let a second block in: rows of 6144 at 5.5 TB/s, 4.3 with 96; of 8192 4.5 and 4.9.
template <typename T>
cudaError_t launch_residual(const ResidualNormArgs &A, int n_sm, cudaLaunchConfig_t &cfg) {
  const int chunks = A.H / 8;
  const auto threads = [&](int ch) { return (chunks + ch * 32 - 1) / (ch * 32) * 32; };
  if (chunks > 1024) return launch_chunks<T, 4, 128>(A, threads(4), n_sm, cfg);
  const int t = threads(2);
  if (2 * t * 96 > 65536 && 2 * t * 80 <= 65536) return launch_chunks<T, 2, 80>(A, t, n_sm, cfg);
  return launch_chunks<T, 2, 96>(A, t, n_sm, cfg);
}

cudaError_t done(cudaError_t e) { return e != cudaSuccess ? e : cudaGetLastError(); }

}  // namespace

cudaError_t launch_gated_norm(const GatedNormArgs &A, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  return done(A.dtype == MFD_BF16 ? launch_gated_width<__nv_bfloat16>(A, cfg) : launch_gated_width<__half>(A, cfg));
}

cudaError_t launch_residual_norm(const ResidualNormArgs &A, int n_sm, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  return done(A.dtype == MFD_BF16 ? launch_residual<__nv_bfloat16>(A, n_sm, cfg) : launch_residual<__half>(A, n_sm, cfg));
}

}  // namespace mfd
