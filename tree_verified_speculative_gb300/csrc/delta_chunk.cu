// delta_chunk.cu -- the gated delta rule over many rows: 64 at a time on the
// tensor cores.
//
//   S' = e^g S,  u = beta (v - S'^T k),  S = S' + k u^T,  o = scale S^T q
//
// For the rows i of a chunk, with c_i the sum of g up to i and G = K K^T, the
// updates solve a unit lower triangular system, and what the chunk leaves is one
// product:
//
//   y_i = r_i u_i:  (I + A) y = b,  A_ij = beta_i r_i^2 e^(c_i - c_j) G_ij (j < i),
//                   b_i = beta_i r_i (v_i - e^(c_i) r_i S^T k_i)
//   o_i = scale s_i (e^(c_i) S^T q_i + sum_{j <= i} e^(c_i - c_j) (q_i . k_j) y_j)
//   S  <- e^(c_end) S + sum_j e^(c_end - c_j) k_j y_j^T
//
// where rows of K and Q are held times a power of two that gives them lengths in
// [1, 2), and r_i, s_i are what is left of their factors (the norm's among
// them).
//
// Operands.  The tensor cores take 16-bit factors.  Keys and queries are fp16
// (bf16's 8 bits fit exactly; only elements below 2^-17 of their row lose bits,
// 2^-25 of the row's length at most).  Everything computed (states, right sides,
// the system's inverse, updates) goes in as the sum of two fp16 numbers, 22 bits,
// scaled by a power of two for each column of the state, so that results are
// fp32's: the product of the two low halves is left out (2^-22).  States stay in
// fp32 registers.
//
// A block has one head's state, transposed: a column of the state is a lane of
// tensor memory and a thread of the chain's warpgroup, so that scales, sums and
// the state itself never cross threads.  Two warpgroups:
//   prep   loads the rows, makes G and Q K^T, inverts I + A (it needs no state),
//          a chunk ahead of
//   chain  S^T [K; Q]^T, b, y = (I + A)^-1 b, the state's step, outputs
//
// Columns of a state do not mix, but rows of a chunk do: 0 times what a later
// row holds is no zero where that is a NaN or an infinity.  A chunk in which
// anything is not finite, or leaves fp16's range, is done over row by row from
// the inputs, in fp32, by the same threads.
#include <atomic>

#include "delta.h"
#include "kvcache.h"
#include "mfd_device.cuh"
#include "tc16.cuh"

namespace mfd {
namespace {

constexpr int C = 64;         // rows of a chunk
constexpr int MAX_DK = 128;
constexpr int LANES = 128;    // columns of a state in a block
constexpr int THREADS = 256;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LEAST_LOG = -1e5f;  // of a decay: e^-1e5 is 0 in fp32, and sums of it stay finite

constexpr int BLOCK = 128 * 128;           // 64 columns of the 128 rows of keys and queries
constexpr int TRI = C * 128;               // a 64 x 64 operand
constexpr int PAD = C + 4;                 // floats of a row of the prep's scratch
struct Coef {                              // of a chunk's rows
  float rb[C], rx[C], until[C], ec[C];
};
struct alignas(1024) Stage {
  uint8_t kq[2 * BLOCK];  // keys' 64 rows, then queries': [64-column block][row][128 bytes, swizzled]
  uint8_t th[TRI], tl[TRI], ph[TRI], pl[TRI];
  uint16_t v[C * LANES];
  Coef c;
};
struct Smem {
  Stage st[2];
  float A[C * PAD], T[C * PAD];
  float n2[2 * C];                         // squared lengths
  float chi[C], clo[C], g[C], beta[C];
  float fq[3][C];                          // outputs' factors, which are used a chunk later than the rest
  uint64_t full[2], empty[2], gram, x, xq, u, s, o, drain;
  uint32_t tmem;
  int bad[2], chain_bad, abort;
};
constexpr int SMEM = sizeof(Smem) + 1024;  // and to a 1024-byte border
static_assert(SMEM <= 232448, "shared memory of one CTA");

// Tensor memory, columns.  What is written over what has been read by then.
constexpr int TM_S = 0;      // the state's halves (64 + 64); right sides' (32 + 32); the state's step (128)
constexpr int TM_XK = 128;   // S^T K^T; the updates
constexpr int TM_XQ = 192;   // S^T Q^T, then outputs; two in turn
constexpr int TM_Y = 320;    // the updates' halves (32 + 32)
constexpr int TM_Z = 384;    // the updates' halves times their decays
constexpr int TM_G = 448;    // [K; Q] K^T

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

template <typename T>
__global__ void __launch_bounds__(THREADS, 1) delta_chunk_kernel(const DeltaArgs p, int slices) {
  extern __shared__ uint8_t raw_smem[];
  Smem &sm = *reinterpret_cast<Smem *>(raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % slices, h = blockIdx.x / slices % p.Hv, r = blockIdx.x / slices / p.Hv;
  const int hk = h / (p.Hv / p.Hk);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
      sm.bad[i] = 0;
    }
    mbar_init(&sm.gram, 1);
    mbar_init(&sm.x, 1);
    mbar_init(&sm.xq, 1);
    mbar_init(&sm.u, 1);
    mbar_init(&sm.s, 1);
    mbar_init(&sm.o, 1);
    mbar_init(&sm.drain, 2);
    sm.chain_bad = 0;
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  block_sync();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  // not before the block has its tensor memory: a grid launched from here on may
  // ask for some on the same SM and keep it until this grid has ended
  pdl_launch_dependents();
  pdl_wait();
  const Request q = request(p, r);
  const int nn = q.ok ? q.nn : 0, n_chunk = (nn + C - 1) / C;
  const int64_t tok0 = (int64_t)r * p.N;
  volatile int *abort_flag = &sm.abort;
  bool ok = true;
  // A wait that ran out, or was told to stop, ends the work: every thread goes on
  // through its loop without waiting or touching anything.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity, abort_flag)) {
      ok = false;
      if (!*abort_flag) report(p.status, MFD_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    ok = __all_sync(0xffffffffu, ok);
  };

  if (warp >= 4) {
    // ----------------------------------------------------------- prep
    const int t = tid - 128, c8 = t & 15, r8 = t >> 4;
    uint4 raw[16];
    float graw = 0.f, braw = 0.f;
    // rows r8, r8 + 8, .. of keys, then of queries, 8 columns each; g and beta of row t
    auto load = [&](int n) {
      const int row0 = n * C;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = row0 + (i * 8 + r8) % C;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (row < nn && c8 * 8 < p.Dk)
          raw[i] = __ldg(reinterpret_cast<const uint4 *>((i < 8 ? p.k + (tok0 + row) * p.k_stride : p.q + (tok0 + row) * p.q_stride) +
                                                         hk * p.Dk + c8 * 8));
      }
      graw = braw = 0.f;
      if (t < C && row0 + t < nn) {
        graw = __ldg(p.g + (tok0 + row0 + t) * p.Hv + h);
        braw = __ldg(p.beta + (tok0 + row0 + t) * p.Hv + h);
      }
    };
    if (n_chunk) load(0);
    for (int i = t; i < C * PAD; i += 128) sm.T[i] = 0.f;  // above its diagonal blocks it stays so
    for (int n = 0; n < n_chunk; ++n) {
      Stage &st = sm.st[n & 1];
      wait(&sm.empty[n & 1], ((n >> 1) & 1u) ^ 1u);
      bool bad = false;
      if (t == 0) sm.bad[n & 1] = 0;
      // values, as they are
      for (int i = t; i < C * 16; i += 128) {
        const int row = i >> 4, ch = i & 15, col = slice * LANES + ch * 8;
        uint8_t *dst = reinterpret_cast<uint8_t *>(st.v) + row * (LANES * 2) + ch * 16;
        if (!ok) continue;
        if (n * C + row < nn && col < p.Dv)
          cp_async16(smem_u32(dst), p.v + (tok0 + n * C + row) * p.v_stride + h * p.Dv + col);
        else
          *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
      }
      if (t < C) {
        sm.g[t] = graw < LEAST_LOG ? LEAST_LOG : graw;
        sm.beta[t] = braw;
        if (!finite(braw) || !(graw < INFINITY)) bad = true;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = i * 8 + r8;
        float x[8], ss = 0.f;
        unpack8<T>(raw[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!finite(ss)) bad = true;
        const int half_e = ((int)(__float_as_uint(ss) >> 23) - 127) >> 1;  // floor(log2 of the length)
        const float f = __uint_as_float((uint32_t)(127 - half_e) << 23);
        __half2 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __floats2half2_rn(x[2 * e] * f, x[2 * e + 1] * f);
        if (ok) {
          *reinterpret_cast<uint4 *>(st.kq + (c8 >> 3) * BLOCK + row * 128 + (((c8 & 7) ^ (row & 7)) << 4)) =
              *reinterpret_cast<const uint4 *>(y);
          if (c8 == 0) sm.n2[row] = ss;
        }
      }
      fence_async_smem();
      named_sync(2, 128);
      if (warp == 4) {
        if (elect_one() && ok) {
          tc_fence_after();
          constexpr uint32_t id = idesc_16<__half>(128, C, false);
          const uint32_t a = desc_lo(smem_u32(st.kq), 16);
          const int steps = p.Dk / 16;
          for (int k = 0; k < steps; ++k) {
            const uint32_t at = (k >> 2) * (BLOCK >> 4) + (k & 3) * 2;
            mma_ss(tmem + TM_G, a + at, a + at, id, k != 0);
          }
          tc_commit(&sm.gram);
        }
        __syncwarp();
        // sums of the log decays, in 64 bits, two rows a lane; kept in units of log 2 as two floats
        const double a = (double)sm.g[2 * lane], b = (double)sm.g[2 * lane + 1];
        double run = a + b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double up = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += up;
        }
        const double c1 = run * (double)1.4426950408889634, c0 = (run - b) * (double)1.4426950408889634;
        sm.chi[2 * lane] = (float)c0;
        sm.clo[2 * lane] = (float)(c0 - (double)(float)c0);
        sm.chi[2 * lane + 1] = (float)c1;
        sm.clo[2 * lane + 1] = (float)(c1 - (double)(float)c1);
      }
      if (n + 1 < n_chunk) load(n + 1);
      named_sync(2, 128);
      wait(&sm.gram, n & 1u);
      // this thread's row of [K; Q] K^T
      const int row = t & 63;
      const bool is_q = t >= C;
      const float chi = sm.chi[row], clo = sm.clo[row];
      const float ss = sm.n2[t];
      const int half_e = ((int)(__float_as_uint(ss) >> 23) - 127) >> 1;
      const float left = (p.normalize ? rsqrtf(ss + p.eps) : 1.f) * __uint_as_float((uint32_t)(127 + half_e) << 23);
      const float br = sm.beta[row] * left, brr = br * left;
      if (!is_q) {
        const float ec = ex2(chi + clo);
        const float until = ex2((sm.chi[C - 1] - chi) + (sm.clo[C - 1] - clo));
        st.c.rb[row] = br;
        st.c.rx[row] = -brr * ec;
        st.c.until[row] = until;
        st.c.ec[row] = ec;
        if (!finite(br) || !finite(brr * ec) || !finite(until)) bad = true;
      } else {
        sm.fq[n % 3][row] = left * p.scale;
        if (!finite(left)) bad = true;
      }
      if (ok) {
        tc_fence_after();
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          uint32_t x[32];
          tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + TM_G + part * 32, x);
          tmem_wait_ld();
          tie32(x);
#pragma unroll
          for (int k8 = 0; k8 < 4; ++k8) {
            const int j0 = part * 32 + k8 * 8;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int j = j0 + e;
              const float d = ex2((chi - sm.chi[j]) + (clo - sm.clo[j]));
              const float z = __uint_as_float(x[k8 * 8 + e]) * (is_q ? d : d * brr);
              y[e] = j < row || (is_q && j == row) ? z : 0.f;
              if (!finite(y[e])) bad = true;
            }
            if (is_q) {
              uint4 hi, lo;
              halves(y[0], y[1], hi.x, lo.x);
              halves(y[2], y[3], hi.y, lo.y);
              halves(y[4], y[5], hi.z, lo.z);
              halves(y[6], y[7], hi.w, lo.w);
              const int at = row * 128 + (((j0 >> 3) ^ (row & 7)) << 4);
              *reinterpret_cast<uint4 *>(st.ph + at) = hi;
              *reinterpret_cast<uint4 *>(st.pl + at) = lo;
            } else {
              *reinterpret_cast<float4 *>(&sm.A[row * PAD + j0]) = make_float4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<float4 *>(&sm.A[row * PAD + j0 + 4]) = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
        }
        tc_fence_before();
      }
      named_sync(2, 128);
      // (I + A)^-1: of the four 16 x 16 blocks on the diagonal, a column a thread ..
      if (t < C) {
        const int b = t >> 4, col = t & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float acc = i == col ? 1.f : 0.f;
#pragma unroll
          for (int m = 0; m < i; ++m) acc = fmaf(-sm.A[(16 * b + i) * PAD + 16 * b + m], x[m], acc);
          x[i] = i < col ? 0.f : acc;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) sm.T[(16 * b + i) * PAD + 16 * b + col] = x[i];
      }
      named_sync(2, 128);
      // .. then of blocks twice as large, twice: the lower left part of a pair is
      // -T_below A_left T_above.  A's upper right parts, which nothing reads, hold
      // the first product.
#pragma unroll 1
      for (int size = 16; size <= 32; size *= 2) {
        // a thread's 4 columns of a row: pairs * size * size / 4 of them
        const int quads = size / 4, per = size * quads;
        for (int i = t; i < (C / (2 * size)) * per; i += 128) {
          const int b = i / per * 2 * size, row = i % per / quads, col = i % quads * 4;
          float4 acc = make_float4(0, 0, 0, 0);
          for (int m = 0; m < size; ++m) {
            const float a = sm.A[(b + size + row) * PAD + b + m];
            const float4 x = *reinterpret_cast<const float4 *>(&sm.T[(b + m) * PAD + b + col]);
            acc.x = fmaf(a, x.x, acc.x);
            acc.y = fmaf(a, x.y, acc.y);
            acc.z = fmaf(a, x.z, acc.z);
            acc.w = fmaf(a, x.w, acc.w);
          }
          *reinterpret_cast<float4 *>(&sm.A[(b + row) * PAD + b + size + col]) = acc;
        }
        named_sync(2, 128);
        for (int i = t; i < (C / (2 * size)) * per; i += 128) {
          const int b = i / per * 2 * size, row = i % per / quads, col = i % quads * 4;
          float4 acc = make_float4(0, 0, 0, 0);
          for (int m = 0; m <= row; ++m) {
            const float a = -sm.T[(b + size + row) * PAD + b + size + m];
            const float4 x = *reinterpret_cast<const float4 *>(&sm.A[(b + m) * PAD + b + size + col]);
            acc.x = fmaf(a, x.x, acc.x);
            acc.y = fmaf(a, x.y, acc.y);
            acc.z = fmaf(a, x.z, acc.z);
            acc.w = fmaf(a, x.w, acc.w);
          }
          *reinterpret_cast<float4 *>(&sm.T[(b + size + row) * PAD + b + col]) = acc;
        }
        named_sync(2, 128);
      }
      {
        // its halves: half a row a thread; what lies above the diagonal is zero
        const int row = t >> 1, j1 = (t & 1) * 32;
#pragma unroll
        for (int k8 = 0; k8 < 4; ++k8) {
          const int j0 = j1 + k8 * 8;
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = j0 + e <= row ? sm.T[row * PAD + j0 + e] : 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!(fabsf(y[e]) < 65504.f)) bad = true;
          uint4 hi, lo;
          halves(y[0], y[1], hi.x, lo.x);
          halves(y[2], y[3], hi.y, lo.y);
          halves(y[4], y[5], hi.z, lo.z);
          halves(y[6], y[7], hi.w, lo.w);
          const int at = row * 128 + (((j0 >> 3) ^ (row & 7)) << 4);
          if (ok) {
            *reinterpret_cast<uint4 *>(st.th + at) = hi;
            *reinterpret_cast<uint4 *>(st.tl + at) = lo;
          }
        }
      }
      if (bad) sm.bad[n & 1] = 1;
      cp_async_wait();
      fence_async_smem();
      named_sync(2, 128);
      if (t == 0 && ok) mbar_arrive(&sm.full[n & 1]);
    }
    if (warp == 4) {
      if (elect_one()) tc_commit(&sm.drain);
      __syncwarp();
    }
  } else {
    // ----------------------------------------------------------- chain
    const int col = slice * LANES + tid;
    const bool have = col < p.Dv;
    const uint32_t me = tmem + ((uint32_t)(warp * 32) << 16);
    float s[MAX_DK];
    {
      const float *from = p.s + ((int64_t)q.src * p.Hv + h) * p.Dk * p.Dv + col;
#pragma unroll
      for (int d = 0; d < MAX_DK; ++d) s[d] = q.ok && q.src >= 0 && have && d < p.Dk ? from[(int64_t)d * p.Dv] : 0.f;
    }
    uint16_t *out = p.out + (tok0 * p.Hv + h) * p.Dv + col;
    const int64_t out_row = (int64_t)p.Hv * p.Dv;
    if (!q.ok && tid == 0) report(p.status, MFD_ERR_INPUT);
    if (have)
      for (int i = nn; i < p.N; ++i) out[i * out_row] = 0;

    uint32_t n_x = 0, n_u = 0, n_s = 0, n_o = 0;  // uses of each barrier
    bool pending = false;  // outputs of the chunk before wait in tensor memory
    float out_scale = 0.f;
    uint32_t pending_xq = 0;
    int pending_n = 0;
    // outputs of a chunk that are left: scale s_i times what the products gave
    auto put_outputs = [&]() {
      if (!pending) return;
      pending = false;
      wait(&sm.o, (n_o - 1u) & 1u);
      if (!ok) return;
      tc_fence_after();
      const float *fq = sm.fq[pending_n % 3];
      const int rows = min(C, nn - pending_n * C);
      uint16_t *to = out + (int64_t)pending_n * C * out_row;
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        uint32_t x[32];
        tmem_ld32(me + TM_XQ + pending_xq * C + part * 32, x);
        tmem_wait_ld();
        tie32(x);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float y = __uint_as_float(x[i]) * out_scale * fq[part * 32 + i];
          if (have && part * 32 + i < rows) to[(part * 32 + i) * out_row] = (uint16_t)pack2<T>(y, 0.f);
        }
      }
    };
    // whether any thread of the chain says so; also a barrier
    auto any = [&](bool x) {
      uint32_t y;
      __syncwarp();
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
          "selp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(y)
          : "r"((uint32_t)x)
          : "memory");
      return y != 0;
    };

    for (int n = 0; n < n_chunk; ++n) {
      Stage &st = sm.st[n & 1];
      const uint32_t xq = me + TM_XQ + (n & 1) * C;
      // the state's halves
      float top = 0.f;
#pragma unroll
      for (int d = 0; d < MAX_DK; d += 2) top = max_nan(top, s[d], s[d + 1]);
      float back_s;
      const float up_s = power_for(top, 11, back_s);
      if (ok) {
#pragma unroll
        for (int d = 0; d < MAX_DK; d += 32) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) halves(s[d + 2 * e] * up_s, s[d + 2 * e + 1] * up_s, hi[e], lo[e]);
          tmem_st16(me + TM_S + d / 2, hi);
          tmem_st16(me + TM_S + 64 + d / 2, lo);
        }
        tmem_wait_st();
      }
      wait(&sm.full[n & 1], (n >> 1) & 1u);
      tc_fence_before();
      bool slow = any(!finite(top) || (ok && *(volatile int *)&sm.bad[n & 1]));
      if (!slow) {
        if (warp == 0) {
          if (elect_one() && ok) {
            tc_fence_after();
            constexpr uint32_t id = idesc_16<__half>(128, C, false);
            const int steps = p.Dk / 16;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {  // keys, then queries
              const uint32_t b = desc_lo(smem_u32(st.kq), 16) + half * (C * 128 >> 4);
              const uint32_t d = tmem + (half ? TM_XQ + (n & 1) * C : TM_XK);
              for (int k = 0; k < 2 * steps; ++k) {
                const int kk = k < steps ? k : k - steps;
                mma_ts(d, tmem + TM_S + (k < steps ? 0 : 64) + kk * 8, b + (kk >> 2) * (BLOCK >> 4) + (kk & 3) * 2, id, k != 0);
              }
              tc_commit(half ? &sm.xq : &sm.x);
            }
          }
          __syncwarp();
        }
        put_outputs();
        // right sides
        wait(&sm.x, n_x & 1u);
        tc_fence_after();
        float b[C];
        top = 0.f;
        if (ok) {
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t x[32];
            tmem_ld32(me + TM_XK + part * 32, x);
            tmem_wait_ld();
            tie32(x);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int row = part * 32 + i;
              const float v = to_float<T>(st.v[row * LANES + tid]);
              b[row] = fmaf(st.c.rx[row], __uint_as_float(x[i]) * back_s, st.c.rb[row] * v);
            }
          }
#pragma unroll
          for (int i = 0; i < C; i += 2) top = max_nan(top, b[i], b[i + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < C; ++i) b[i] = 0.f;
        }
        float back_b;
        float up_b = power_for(top, 8, back_b);
        if (up_b > up_s * 0x1p60f) {  // nothing to add: the outputs' common scale stays near the state's
          up_b = up_s * 0x1p60f;
          back_b = back_s * 0x1p-60f;
        }
        wait(&sm.xq, n_x & 1u);  // the state's halves have been read
        ++n_x;
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < C; i += 32) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) halves(b[i + 2 * e] * up_b, b[i + 2 * e + 1] * up_b, hi[e], lo[e]);
            tmem_st16(me + TM_S + i / 2, hi);
            tmem_st16(me + TM_S + 32 + i / 2, lo);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        slow = any(!finite(top));
        if (!slow) {
          if (warp == 0) {
            if (elect_one() && ok) {
              tc_fence_after();
              constexpr uint32_t id = idesc_16<__half>(128, C, false);
              const uint32_t th = desc_lo(smem_u32(st.th), 16), tl = desc_lo(smem_u32(st.tl), 16);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ts(tmem + TM_XK, tmem + TM_S + k * 8, th + k * 2, id, k != 0);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ts(tmem + TM_XK, tmem + TM_S + 32 + k * 8, th + k * 2, id, 1);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ts(tmem + TM_XK, tmem + TM_S + k * 8, tl + k * 2, id, 1);
              tc_commit(&sm.u);
            }
            __syncwarp();
          }
          // meanwhile the outputs' first part, to the updates' scale
          if (ok) {
            const float f = up_b * back_s;
#pragma unroll
            for (int part = 0; part < 4; ++part) {
              uint32_t x[16];
              tmem_ld16(xq + part * 16, x);
              tmem_wait_ld();
              tie16(x);
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f * st.c.ec[part * 16 + i]);
              tmem_st16(xq + part * 16, x);
            }
          }
          // the updates
          wait(&sm.u, n_u & 1u);
          ++n_u;
          if (ok) {
            tc_fence_after();
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t x[32];
              tmem_ld32(me + TM_XK + part * 32, x);
              tmem_wait_ld();
              tie32(x);
#pragma unroll
              for (int i = 0; i < 32; ++i) b[part * 32 + i] = __uint_as_float(x[i]);
            }
            top = 0.f;
#pragma unroll
            for (int i = 0; i < C; i += 2) top = max_nan(top, b[i], b[i + 1]);
#pragma unroll
            for (int i = 0; i < C; i += 32) {
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                halves(b[i + 2 * e] * st.c.until[i + 2 * e], b[i + 2 * e + 1] * st.c.until[i + 2 * e + 1], hi[e], lo[e]);
              tmem_st16(me + TM_Z + i / 2, hi);
              tmem_st16(me + TM_Z + 32 + i / 2, lo);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          slow = any(!(top < 65504.f));
          if (!slow) {
            if (warp == 0) {
              if (elect_one() && ok) {
                tc_fence_after();
                constexpr uint32_t id = idesc_16<__half>(128, 128, true);
                const uint32_t kd = desc_lo(smem_u32(st.kq), BLOCK);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  mma_ts(tmem + TM_S, tmem + TM_Z + (k >> 2) * 32 + (k & 3) * 8, kd + (k & 3) * (2048 >> 4), id, k != 0);
                tc_commit(&sm.s);
              }
              __syncwarp();
            }
            if (ok) {
#pragma unroll
              for (int i = 0; i < C; i += 32) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) halves(b[i + 2 * e], b[i + 2 * e + 1], hi[e], lo[e]);
                tmem_st16(me + TM_Y + i / 2, hi);
                tmem_st16(me + TM_Y + 32 + i / 2, lo);
              }
              tmem_wait_st();
            }
            const float d = st.c.ec[C - 1];
            tc_fence_before();
            named_sync(1, 128);
            if (warp == 0) {
              if (elect_one() && ok) {
                tc_fence_after();
                constexpr uint32_t id = idesc_16<__half>(128, C, false);
                const uint32_t ph = desc_lo(smem_u32(st.ph), 16), pl = desc_lo(smem_u32(st.pl), 16);
                const uint32_t d = tmem + TM_XQ + (n & 1) * C;
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ts(d, tmem + TM_Y + k * 8, ph + k * 2, id, 1);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ts(d, tmem + TM_Y + 32 + k * 8, ph + k * 2, id, 1);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ts(d, tmem + TM_Y + k * 8, pl + k * 2, id, 1);
                tc_commit(&sm.o);
                tc_commit(&sm.empty[n & 1]);  // all that reads this stage is done by then
              }
              __syncwarp();
            }
            ++n_o;
            pending = true;
            pending_xq = n & 1;
            pending_n = n;
            out_scale = back_b;
            wait(&sm.s, n_s & 1u);
            ++n_s;
            if (ok) {
              tc_fence_after();
#pragma unroll
              for (int part = 0; part < 4; ++part) {
                uint32_t x[32];
                tmem_ld32(me + TM_S + part * 32, x);
                tmem_wait_ld();
                tie32(x);
#pragma unroll
                for (int i = 0; i < 32; ++i) s[part * 32 + i] = fmaf(s[part * 32 + i], d, __uint_as_float(x[i]) * back_b);
              }
            }
          }
        }
      }
      if (slow) {
        // row by row from the inputs, as delta_rows.cu does it
        put_outputs();
        const int rows = min(C, nn - n * C);
#pragma unroll 1
        for (int i = 0; i < rows; ++i) {
          const int64_t tok = tok0 + n * C + i;
          const uint4 *kr = reinterpret_cast<const uint4 *>(p.k + tok * p.k_stride + hk * p.Dk);
          const uint4 *qr = reinterpret_cast<const uint4 *>(p.q + tok * p.q_stride + hk * p.Dk);
          float fk = 1.f, fq = 1.f, x[8], y[8];
          if (p.normalize) {
            float a = 0.f, b = 0.f;
#pragma unroll 1
            for (int c = 0; c < p.Dk / 8; ++c) {
              unpack8<T>(__ldg(kr + c), x);
              unpack8<T>(__ldg(qr + c), y);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                a = fmaf(x[e], x[e], a);
                b = fmaf(y[e], y[e], b);
              }
            }
            fk = rsqrtf(a + p.eps);
            fq = rsqrtf(b + p.eps);
          }
          float ks = 0.f, qs = 0.f, kq = 0.f;
#pragma unroll
          for (int c = 0; c < MAX_DK / 8; ++c)
            if (c * 8 < p.Dk) {
              unpack8<T>(__ldg(kr + c), x);
              unpack8<T>(__ldg(qr + c), y);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float k = x[e] * fk, qq = y[e] * fq;
                ks = fmaf(k, s[c * 8 + e], ks);
                qs = fmaf(qq, s[c * 8 + e], qs);
                kq = fmaf(k, qq, kq);
              }
            }
          const float d = expf(__ldg(p.g + tok * p.Hv + h)), beta = __ldg(p.beta + tok * p.Hv + h);
          const float v = have ? to_float<T>(p.v[tok * p.v_stride + h * p.Dv + col]) : 0.f;
          const float u = beta * fmaf(-d, ks, v);
#pragma unroll
          for (int c = 0; c < MAX_DK / 8; ++c)
            if (c * 8 < p.Dk) {
              unpack8<T>(__ldg(kr + c), x);
#pragma unroll
              for (int e = 0; e < 8; ++e) s[c * 8 + e] = fmaf(x[e] * fk, u, d * s[c * 8 + e]);
            }
          if (have) out[(n * C + i) * out_row] = (uint16_t)pack2<T>(p.scale * fmaf(kq, u, d * qs), 0.f);
        }
        named_sync(1, 128);  // all have read the stage
        if (warp == 0) {
          if (elect_one() && ok) tc_commit(&sm.empty[n & 1]);
          __syncwarp();
        }
      }
    }
    put_outputs();
    if (ok && q.ok && q.dst >= 0 && have) {
      float *to = p.s + ((int64_t)q.dst * p.Hv + h) * p.Dk * p.Dv + col;
#pragma unroll
      for (int d = 0; d < MAX_DK; ++d)
        if (d < p.Dk) to[(int64_t)d * p.Dv] = s[d];
    }
    if (warp == 0) {  // no product runs on when tensor memory is given back
      if (elect_one()) {
        tc_commit(&sm.drain);
        int never = 0;
        mbar_wait(&sm.drain, 0, &never);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  block_sync();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <typename T>
cudaError_t launch_type(const DeltaArgs &A, cudaStream_t stream) {
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};  // devices this kernel is set up on
  if (dev > 63 || !((ready.load(std::memory_order_relaxed) >> dev) & 1u)) {
    if ((e = cudaFuncSetAttribute(delta_chunk_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM)) != cudaSuccess)
      return e;
    if (dev < 64) ready.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  }
  const int slices = (A.Dv + LANES - 1) / LANES;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)A.n_req * A.Hv * slices));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  e = cudaLaunchKernelEx(&cfg, delta_chunk_kernel<T>, A, slices);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaArgs &A, cudaStream_t stream) {
  return A.dtype == MFD_BF16 ? launch_type<__nv_bfloat16>(A, stream) : launch_type<__half>(A, stream);
}

}  // namespace mfd
