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
// where k_j and q_i are taken times a power of two that gives them lengths in
// [1, 2) (2^40 at most), and r_i, s_i are what is left of their factors (the norm's among them).
//
// Operands.  The tensor cores take 16-bit factors.  Keys and queries go in as
// they are; their powers are in the other factors.  The state, and what its step
// takes of the updates, go in as sums of numbers of their type: three of bf16,
// each the front of what is left (24 bits), or two of fp16 after a power of two
// for each column, which brings its largest to [2^14, 2^15) (22 bits of what is at
// least 2^-17 of that; 2^-39 of the largest below).  What meets no key or query (the right sides, the
// system's inverse, P, the updates) is three bf16 numbers, each row's as exact as
// if it were alone: rows of a chunk differ in size by whatever their values, steps
// and decays do, and two fp16 numbers under a power of two for a column took from
// the small ones what the largest, a later one too, left no room for.  Six of the
// nine products of two such sums are made, smallest first; what the others leave
// out is 2^-24 of a term on average, and below 2^-21.  So results are fp32's.  The
// state itself stays in fp32 registers: the tensor cores' sums cut off what they
// cannot hold, and a step added to it there, sixteen rows at a time, left slow heads'
// states 3e-6 off after some thousand rows.
//
// A block has one head's state, transposed: a column of the state is a lane of
// tensor memory, which two threads of the chain share, half of the column and
// half of a chunk's rows each.  Scales, sums and the state itself never cross
// columns.  Eight warps each (more would leave too few registers):
//   prep   loads the rows, makes K K^T and Q K^T, inverts I + A (it needs no
//          state), a chunk ahead of
//   chain  S^T [K; Q]^T, b, y = (I + A)^-1 b, the state's step, outputs
//
// Columns of a state do not mix, but rows of a chunk do: 0 times what a later
// row holds is no zero where that is a NaN or an infinity.  A chunk in which
// anything is not finite, or grows as no working layer's does, is done over row
// by row from the inputs, in fp32, by the chain's threads.
//
// A prompt of 4001 rows and 32 heads of 128 x 128 takes 432 us: 13,300 cycles a chunk,
// which prep and chain both need, each a line of phases that wait for one another, and
// 32 of the SMs have work.  Eight prompts of 975 to 2000 rows take 386 us.  (In fp16 437
// and 366; with two fp16 numbers for the right sides, the inverse and the updates 416 and
// 367 in bf16.)
#include <atomic>
#include <type_traits>

#include "delta_tc.cuh"

namespace mfd {
namespace {

constexpr int C = 64;         // rows of a chunk
constexpr int MAX_DK = 128;
constexpr int LANES = 128;    // columns of a state in a block
constexpr int CHAIN = 256, PREP = 256, THREADS = CHAIN + PREP;
// Largest elements of a chunk, past which it goes row by row: of the inverse and of P (unit
// keys and steps up to 1 leave 1), of S^T K^T and the right sides (past it what a product
// of decays below fp32's smallest takes with it may count), and of the updates' factors in
// the step.  Within them all that follows is finite.
constexpr float MOST = 0x1p16f, MOST_SUM = 0x1p60f, MOST_UNTIL = 0x1p40f;
// Registers of the two roles' threads: what the one gives up the other takes.
constexpr int LAUNCH_REGS = 128, PREP_REGS = 96, CHAIN_REGS = 160;
static_assert(PREP * PREP_REGS + CHAIN * CHAIN_REGS == THREADS * LAUNCH_REGS && THREADS * LAUNCH_REGS == 65536, "registers of an SM");

constexpr int BLOCK = 128 * 128;           // 64 columns of the 128 rows of keys and queries
constexpr int TRI = C * 128;               // a 64 x 64 operand
constexpr int PAD = C + 4;                 // floats of a row of the prep's scratch
struct Coef {                              // of a chunk's rows
  float2 rhs[C];                           // of v and of S^T k in b
  float until[C], eq[C], end;              // of the updates in the step, of S^T q in o, of the state
};
struct alignas(1024) Stage {
  uint8_t kq[2 * BLOCK];  // keys' 64 rows, then queries': [64-column block][row][128 bytes, swizzled]
  uint8_t p3[3][TRI];     // P's parts
  uint16_t v[C * LANES];
};
struct Smem {
  Stage st[2];
  uint8_t t3[3][TRI];                      // the inverse's parts, of one chunk
  Coef c[2];
  float At[C * PAD], T[C * PAD];           // A transposed; the inverse
  uint16_t out[C * LANES];
  float n2[2 * C];                         // squared lengths
  float4 cc[C];                            // sums of log2 decays as two floats each; the key's power
  float g[C], beta[C];
  float fq[3][C];                          // outputs' factors, which are used a chunk later than the rest
  float top[2][2][LANES];                  // [state, right sides][half][column]
  uint64_t full[2], empty[2], gram, x, xq, u, s, o, drain, ps, pq, pb, pz, py;
  uint32_t tmem;
  int bad[2], chain_bad, abort, request;
};
constexpr int SMEM = sizeof(Smem) + 1024;  // and to a 1024-byte border
static_assert(SMEM <= 232448, "shared memory of one CTA");

// Tensor memory, columns.  What is written over what has been read by then.
constexpr int TM_S = 0;      // the state's step
constexpr int TM_H = 128;    // the state's parts (64 each); right sides' parts (32 each), then the updates'
constexpr int TM_Z = 224;    // the parts of the updates times their decays (32 each)
constexpr int TM_XK = 320;   // S^T K^T; the updates
constexpr int TM_XQ = 384;   // S^T Q^T, then outputs
constexpr int TM_G = 448;    // [K; Q] K^T

// Three bf16 numbers of two floats: each the front of what is left.
__device__ __forceinline__ void thirds(float a, float b, uint32_t &x, uint32_t &y, uint32_t &z) {
  x = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  a -= __uint_as_float(x << 16);
  b -= __uint_as_float(x & 0xFFFF0000u);
  y = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  a -= __uint_as_float(y << 16);
  b -= __uint_as_float(y & 0xFFFF0000u);
  z = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

// floor(log2 of the length) from its square, at least -40: of a key that short the powers
// would leave MOST_UNTIL.  Of a key of zeros, which no power makes longer, 0.
__device__ __forceinline__ int length_exponent(float len2) {
  return max(((int)(__float_as_uint(len2 > 0.f ? len2 : 1.f) >> 23) - 127) >> 1, -40);
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 1) delta_chunk_kernel(const DeltaArgs p, int slices) {
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int PARTS = BF16 ? 3 : 2;
  extern __shared__ uint8_t raw_smem[];
  Smem &sm = *reinterpret_cast<Smem *>(raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % slices, h = blockIdx.x / slices % p.Hv;
  const int hk = h / (p.Hv / p.Hk);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 2);
      sm.bad[i] = 0;
    }
    for (uint64_t *b : {&sm.gram, &sm.x, &sm.xq, &sm.u, &sm.s, &sm.o}) mbar_init(b, 1);
    for (uint64_t *b : {&sm.ps, &sm.pq, &sm.pb, &sm.pz, &sm.py}) mbar_init(b, CHAIN / 32);
    mbar_init(&sm.drain, 6);
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
  // The longest requests' blocks come first (while a thread a request orders them): a
  // short one's fit where the long ones leave SMs free at the end.
  int r = blockIdx.x / slices / p.Hv;
  if (p.n_nodes && p.n_req > 1 && p.n_req <= THREADS) {
    int *len = reinterpret_cast<int *>(sm.At);
    const int own = tid < p.n_req ? __ldg(p.n_nodes + tid) : 0;
    if (tid < p.n_req) len[tid] = own;
    block_sync();
    if (tid < p.n_req) {
      int place = 0;
      for (int i = 0; i < p.n_req; ++i) place += len[i] > own || (len[i] == own && i < tid);
      if (place == r) sm.request = tid;
    }
    block_sync();
    r = sm.request;
  }
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
  };
  auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
    wait(bar, parity);
    ok = __all_sync(0xffffffffu, ok);
  };

  if (warp >= CHAIN / 32) {
    // ----------------------------------------------------------- prep
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PREP_REGS));
    const int t = tid - CHAIN;
    for (int i = t; i < C * PAD; i += PREP) sm.T[i] = 0.f;  // above its diagonal blocks it stays so
    for (int n = 0; n < n_chunk; ++n) {
      Stage &st = sm.st[n & 1];
      Coef &cf = sm.c[n & 1];
      const int row0 = n * C;
      wait_warp(&sm.empty[n & 1], ((n >> 1) & 1u) ^ 1u);
      float most = 0.f;  // largest magnitude, NaN where there is one
      bool bad = false;
      if (t == 0) sm.bad[n & 1] = 0;
      // keys, queries and values as they are, zeros past the end
      {
        const int c8 = t & 15, r16 = t >> 4;
        const int64_t tok = tok0 + row0 + r16;
        const uint16_t *kr = p.k + tok * p.k_stride + hk * p.Dk + c8 * 8, *qr = p.q + tok * p.q_stride + hk * p.Dk + c8 * 8;
        const uint16_t *vr = p.v + tok * p.v_stride + h * p.Dv + slice * LANES + c8 * 8;
        const bool dk = c8 * 8 < p.Dk, dv = slice * LANES + c8 * 8 < p.Dv;
        const uint32_t to = smem_u32(st.kq) + (c8 >> 3) * BLOCK + r16 * 128 + (((c8 & 7) ^ (r16 & 7)) << 4);
        const uint32_t tv = smem_u32(st.v) + r16 * (LANES * 2) + c8 * 16;
        if (ok)
#pragma unroll
          for (int i = 0; i < C / 16; ++i) {
            const bool live = row0 + i * 16 + r16 < nn;
            if (live && dk) {
              cp_async16(to + i * (16 * 128), kr + i * 16 * p.k_stride);
              cp_async16(to + (C + i * 16) * 128, qr + i * 16 * p.q_stride);
            } else {
              st_shared16(to + i * (16 * 128), make_uint4(0, 0, 0, 0));
              st_shared16(to + (C + i * 16) * 128, make_uint4(0, 0, 0, 0));
            }
            if (live && dv)
              cp_async16(tv + i * (16 * LANES * 2), vr + i * 16 * p.v_stride);
            else
              st_shared16(tv + i * (16 * LANES * 2), make_uint4(0, 0, 0, 0));
          }
      }
      if (t < C) {
        float g = 0.f, beta = 0.f;
        if (row0 + t < nn) {
          g = __ldg(p.g + (tok0 + row0 + t) * p.Hv + h);
          beta = __ldg(p.beta + (tok0 + row0 + t) * p.Hv + h);
        }
        if (!finite(beta) || !(g < INFINITY)) bad = true;
        sm.g[t] = g < LEAST_LOG ? LEAST_LOG : g;
        sm.beta[t] = beta;
      }
      cp_async_wait();
      fence_async_smem();
      named_sync(2, PREP);
      if (warp == CHAIN / 32) {
        if (elect_one() && ok) {
          tc_fence_after();
          constexpr uint32_t id = idesc_16<T>(128, C, false);
          const uint32_t a = desc_lo(smem_u32(st.kq), 16);
          const int steps = p.Dk / 16;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < steps) {
              const uint32_t at = (k >> 2) * (BLOCK >> 4) + (k & 3) * 2;
              mma_ss(tmem + TM_G, a + at, a + at, id, k != 0);
            }
          tc_commit(&sm.gram);
        }
        __syncwarp();
      } else if (warp == CHAIN / 32 + 1) {
        // sums of the log decays in units of log 2, two rows a lane, as two floats each
        const Two a = two_product(sm.g[2 * lane], LOG2E_HI, LOG2E_LO), b = two_product(sm.g[2 * lane + 1], LOG2E_HI, LOG2E_LO);
        const Two own = two_sum(a, b);
        Two run = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const Two up = {__shfl_up_sync(0xffffffffu, run.hi, o), __shfl_up_sync(0xffffffffu, run.lo, o)};
          if (lane >= o) run = two_sum(up, run);
        }
        Two before = {__shfl_up_sync(0xffffffffu, run.hi, 1), __shfl_up_sync(0xffffffffu, run.lo, 1)};
        if (lane == 0) before = {0.f, 0.f};
        const Two first = two_sum(before, a);
        *reinterpret_cast<float2 *>(&sm.cc[2 * lane]) = make_float2(first.hi, first.lo);
        *reinterpret_cast<float2 *>(&sm.cc[2 * lane + 1]) = make_float2(run.hi, run.lo);
      }
      {  // squared lengths, two threads a row
        const int row = t >> 1, part = t & 1;
        float ss[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x[8];
          unpack8<T>(ld_shared16(smem_u32(st.kq) + part * BLOCK + row * 128 + ((e ^ (row & 7)) << 4)), x);
#pragma unroll
          for (int k = 0; k < 8; ++k) ss[k & 3] = fmaf(x[k], x[k], ss[k & 3]);
        }
        float len2 = (ss[0] + ss[1]) + (ss[2] + ss[3]);
        len2 += __shfl_xor_sync(0xffffffffu, len2, 1);
        if (!finite(len2)) bad = true;
        if (part == 0) {
          sm.n2[row] = len2;
          if (row < C) sm.cc[row].z = __uint_as_float((uint32_t)(127 - length_exponent(len2)) << 23);
        }
      }
      named_sync(2, PREP);
      wait_warp(&sm.gram, n & 1u);
      // this thread's row of [K; Q] K^T, half of its columns
      const int row = t & 63, j1 = (t >> 7) * 32;
      const bool is_q = (t & 127) >= C;
      const float4 ci = sm.cc[row];
      const float len2 = row0 + row < nn ? sm.n2[t & 127] : 1.f;
      const int half_e = length_exponent(len2);
      const float left = (p.normalize ? rsqrtf(len2 + p.eps) : 1.f) * __uint_as_float((uint32_t)(127 + half_e) << 23);
      const float power = __uint_as_float((uint32_t)(127 - half_e) << 23);
      const float br = sm.beta[row] * left, brr = br * left;
      if (t < 2 * C) {
        const float ec = ex2(ci.x + ci.y);
        if (!is_q) {
          const float4 end = sm.cc[C - 1];
          const float until = ex2((end.x - ci.x) + (end.y - ci.y)) * power;
          cf.rhs[row] = make_float2(br, -brr * ec * power);
          cf.until[row] = until;
          if (row == C - 1) cf.end = ec;
          if (!finite(br) || !finite(brr * ec * power) || !(until <= MOST_UNTIL)) bad = true;
        } else {
          cf.eq[row] = ec * power;
          sm.fq[n % 3][row] = left * p.scale;
          if (!finite(left) || !finite(ec)) bad = true;
        }
      }
      if (ok) {
        tc_fence_after();
        uint32_t x[32];
        tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + TM_G + j1, x);
        tmem_wait_ld();
        tie32(x);
        tc_fence_before();
        const float f = is_q ? power : brr * power;
        const int last = is_q ? row : row - 1;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float4 cj = sm.cc[j1 + e];
          const float z = __uint_as_float(x[e]) * (f * (cj.z * ex2((ci.x - cj.x) + (ci.y - cj.y))));
          x[e] = j1 + e <= last ? __float_as_uint(z) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) most = max_nan(most, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        if (is_q) {
#pragma unroll
          for (int k8 = 0; k8 < 4; ++k8) {
            uint32_t y[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              thirds(__uint_as_float(x[k8 * 8 + 2 * e]), __uint_as_float(x[k8 * 8 + 2 * e + 1]), y[0][e], y[1][e], y[2][e]);
            const int at = row * 128 + ((((j1 >> 3) + k8) ^ (row & 7)) << 4);
#pragma unroll
            for (int e = 0; e < 3; ++e) *reinterpret_cast<uint4 *>(st.p3[e] + at) = make_uint4(y[e][0], y[e][1], y[e][2], y[e][3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) sm.At[(j1 + e) * PAD + row] = __uint_as_float(x[e]);
        }
      }
      named_sync(2, PREP);
      // (I + A)^-1: of the four 16 x 16 blocks on the diagonal, a column a thread: an
      // element that is known goes out to all below it ..
      if ((warp & 3) == 2) {
        const int b = (t >> 7) * 32 + (lane & 16), col = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 15; ++m)
#pragma unroll
          for (int i = (m + 1) & ~3; i < 16; i += 4) {  // A is 0 on and above its diagonal
            const float4 a = *reinterpret_cast<const float4 *>(&sm.At[(b + m) * PAD + b + i]);
            x[i] = fmaf(-a.x, x[m], x[i]);
            x[i + 1] = fmaf(-a.y, x[m], x[i + 1]);
            x[i + 2] = fmaf(-a.z, x[m], x[i + 2]);
            x[i + 3] = fmaf(-a.w, x[m], x[i + 3]);
          }
#pragma unroll
        for (int i = 0; i < 16; ++i) sm.T[(b + i) * PAD + b + col] = x[i];
      }
      named_sync(2, PREP);
      // .. then of blocks twice as large, twice: the lower left part of a pair is
      // -T_22 A_21 T_11.  The first product goes where A's transpose has its empty
      // block.
      {
        const int b = (t >> 7) * 32, i = b + 16 + ((t & 127) >> 3), j = b + (t & 7) * 2;
        float2 acc = make_float2(0, 0);
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          const float a = sm.At[(b + m) * PAD + i];
          const float2 x = *reinterpret_cast<const float2 *>(&sm.T[(b + m) * PAD + j]);
          acc.x = fmaf(a, x.x, acc.x);
          acc.y = fmaf(a, x.y, acc.y);
        }
        *reinterpret_cast<float2 *>(&sm.At[i * PAD + j]) = acc;
        named_sync(2, PREP);
        acc = make_float2(0, 0);
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
          const float4 a = *reinterpret_cast<const float4 *>(&sm.T[i * PAD + b + 16 + m]);
          const float aa[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = *reinterpret_cast<const float2 *>(&sm.At[(b + 16 + m + e) * PAD + j]);
            acc.x = fmaf(-aa[e], x.x, acc.x);
            acc.y = fmaf(-aa[e], x.y, acc.y);
          }
        }
        *reinterpret_cast<float2 *>(&sm.T[i * PAD + j]) = acc;
      }
      named_sync(2, PREP);
      if (t < 128) {  // eight elements a thread, two rows: a load for every five products
        const int i = 32 + (t >> 3) * 2, j = (t & 7) * 4;
        float4 acc[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
#pragma unroll 8
        for (int m = 0; m < 32; ++m) {
          const float2 a = *reinterpret_cast<const float2 *>(&sm.At[m * PAD + i]);
          const float4 x = *reinterpret_cast<const float4 *>(&sm.T[m * PAD + j]);
          acc[0].x = fmaf(a.x, x.x, acc[0].x);
          acc[0].y = fmaf(a.x, x.y, acc[0].y);
          acc[0].z = fmaf(a.x, x.z, acc[0].z);
          acc[0].w = fmaf(a.x, x.w, acc[0].w);
          acc[1].x = fmaf(a.y, x.x, acc[1].x);
          acc[1].y = fmaf(a.y, x.y, acc[1].y);
          acc[1].z = fmaf(a.y, x.z, acc[1].z);
          acc[1].w = fmaf(a.y, x.w, acc[1].w);
        }
        *reinterpret_cast<float4 *>(&sm.At[i * PAD + j]) = acc[0];
        *reinterpret_cast<float4 *>(&sm.At[(i + 1) * PAD + j]) = acc[1];
        named_sync(9, 128);
        acc[0] = acc[1] = make_float4(0, 0, 0, 0);
#pragma unroll 2
        for (int m = 0; m < 32; m += 4) {
          const float4 a0 = *reinterpret_cast<const float4 *>(&sm.T[i * PAD + 32 + m]);
          const float4 a1 = *reinterpret_cast<const float4 *>(&sm.T[(i + 1) * PAD + 32 + m]);
          const float a[2][4] = {{a0.x, a0.y, a0.z, a0.w}, {a1.x, a1.y, a1.z, a1.w}};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 x = *reinterpret_cast<const float4 *>(&sm.At[(32 + m + e) * PAD + j]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              acc[k].x = fmaf(-a[k][e], x.x, acc[k].x);
              acc[k].y = fmaf(-a[k][e], x.y, acc[k].y);
              acc[k].z = fmaf(-a[k][e], x.z, acc[k].z);
              acc[k].w = fmaf(-a[k][e], x.w, acc[k].w);
            }
          }
        }
        *reinterpret_cast<float4 *>(&sm.T[i * PAD + j]) = acc[0];
        *reinterpret_cast<float4 *>(&sm.T[(i + 1) * PAD + j]) = acc[1];
      }
      named_sync(2, PREP);
      if (n) wait_warp(&sm.u, (n - 1) & 1u);  // the chunk before is done with its own
      {
        // its parts: a quarter of a row a thread
        const int i = t >> 2, j1 = (t & 3) * 16;
#pragma unroll
        for (int k8 = 0; k8 < 2; ++k8) {
          const int j0 = j1 + k8 * 8;
          const float4 a = *reinterpret_cast<const float4 *>(&sm.T[i * PAD + j0]);
          const float4 b = *reinterpret_cast<const float4 *>(&sm.T[i * PAD + j0 + 4]);
          most = max_nan(most, a.x, a.y);
          most = max_nan(most, a.z, a.w);
          most = max_nan(most, b.x, b.y);
          most = max_nan(most, b.z, b.w);
          uint4 x, y, z;
          thirds(a.x, a.y, x.x, y.x, z.x);
          thirds(a.z, a.w, x.y, y.y, z.y);
          thirds(b.x, b.y, x.z, y.z, z.z);
          thirds(b.z, b.w, x.w, y.w, z.w);
          const int at = i * 128 + (((j0 >> 3) ^ (i & 7)) << 4);
          if (ok) {
            *reinterpret_cast<uint4 *>(sm.t3[0] + at) = x;
            *reinterpret_cast<uint4 *>(sm.t3[1] + at) = y;
            *reinterpret_cast<uint4 *>(sm.t3[2] + at) = z;
          }
        }
      }
      if (bad || !(most < MOST)) sm.bad[n & 1] = 1;
      fence_async_smem();
      named_sync(2, PREP);
      if (t == 0 && ok) mbar_arrive(&sm.full[n & 1]);
    }
  } else {
    // ----------------------------------------------------------- chain
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(CHAIN_REGS));
    // A thread has rows 64 half .. of its column of the state, and rows 32 half ..
    // of a chunk.
    constexpr int SD = MAX_DK / 2, SC = C / 2;
    const int half = warp >> 2, l = tid & 127;  // column in the block
    const int d0 = half * SD, i0 = half * SC;
    const int col = slice * LANES + l;
    const bool have = col < p.Dv;
    const uint32_t me = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float s[SD];
    {
      const float *from = p.s + (((int64_t)q.src * p.Hv + h) * p.Dk + d0) * p.Dv + col;
#pragma unroll
      for (int d = 0; d < SD; ++d) s[d] = q.ok && q.src >= 0 && have && d0 + d < p.Dk ? from[(int64_t)d * p.Dv] : 0.f;
    }
    if (!q.ok && tid == 0) report(p.status, MFD_ERR_INPUT);
    {  // rows that are not live
      const int ch = tid & 15;
      if (slice * LANES + ch * 8 < p.Dv)
        for (int i = nn + (tid >> 4); i < p.N; i += CHAIN / 16)
          st_global16(p.out + ((tok0 + i) * p.Hv + h) * p.Dv + slice * LANES + ch * 8, make_uint4(0, 0, 0, 0));
    }
    int pending = -1;  // chunk whose outputs wait in tensor memory
    auto arrive = [&](uint64_t *bar) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(bar);
    };
    // Outputs of that chunk: scale s_i times what the products gave, through shared
    // memory for whole 16 bytes (two bytes a lane took 6,000 cycles a chunk).
    // `next`: the products of the chunk after may go over them once they are read.
    auto put_outputs = [&](bool next) {
      if (pending < 0) {
        if (next) arrive(&sm.pq);
        return;
      }
      wait_warp(&sm.o, pending & 1u);
      const float *fq = sm.fq[pending % 3];
      if (ok) {
        tc_fence_after();
        uint32_t x[SC];
        tmem_ld32(me + TM_XQ + i0, x);
        tmem_wait_ld();
        tie32(x);
        if (next) arrive(&sm.pq);
        // all that is read before all that is written: a load does not pass a store
#pragma unroll
        for (int i = 0; i < SC; ++i) x[i] = pack2<T>(__uint_as_float(x[i]) * fq[i0 + i], 0.f);
#pragma unroll
        for (int i = 0; i < SC; ++i) sm.out[(i0 + i) * LANES + l] = (uint16_t)x[i];
      }
      named_sync(3 + half, 128);
      const int rows = nn - pending * C, ch = l & 15;
      if (ok && slice * LANES + ch * 8 < p.Dv) {
        uint4 y[SC / 8];
#pragma unroll
        for (int k = 0; k < SC / 8; ++k) y[k] = *reinterpret_cast<const uint4 *>(&sm.out[(i0 + k * 8 + (l >> 4)) * LANES + ch * 8]);
        uint16_t *to = p.out + ((tok0 + pending * C + i0 + (l >> 4)) * p.Hv + h) * p.Dv + slice * LANES + ch * 8;
#pragma unroll
        for (int k = 0; k < SC / 8; ++k)
          if (i0 + k * 8 + (l >> 4) < rows) st_global16(to + (int64_t)k * 8 * p.Hv * p.Dv, y[k]);
      }
      pending = -1;
    };
    // the larger of this thread's and the column's other thread's
    auto of_both = [&](int which, float x) {
      sm.top[which][half][l] = x;
      named_sync(5 + (warp & 3), 64);
      return max_nan(x, sm.top[which][half ^ 1][l], 0.f);
    };
    // Whether any thread of the chain says so.
    auto any = [&](bool x) {
      uint32_t y;
      __syncwarp();
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
          "selp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(y)
          : "r"((uint32_t)x), "n"(CHAIN)
          : "memory");
      return y != 0;
    };
    constexpr uint32_t id_t = idesc_16<T>(128, C, false), id_kd = idesc_16<T>(128, 128, true);
    const int steps = p.Dk / 16;
    // Products: one lane of warp `who` issues them once all of the chain's warps have
    // arrived; a warp for each kind, so that none is held up for long.
    auto products = [&](int who, uint64_t *ready, uint32_t par, auto issue) {
      if (warp != who) return;
      wait_warp(ready, par);
      if (elect_one() && ok) {
        tc_fence_after();
        issue();
      }
      __syncwarp();
    };

    // D (+)= A B^T of two sums of three bf16 numbers, rows of A in tensor memory (TM_H), B
    // lower triangular: places 16 k .. have nothing for the rows before 16 k.
    auto triangle = [&](uint32_t d, const uint8_t (&b3)[3][TRI], bool add) {
      constexpr int A[6] = {0, 1, 2, 0, 1, 0}, B[6] = {2, 1, 0, 1, 0, 0};  // smallest first
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        const uint32_t b = desc_lo(smem_u32(b3[B[i]]), 16);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(tmem + d + k * 16, tmem + TM_H + A[i] * 32 + k * 8, b + (k * 16 * 128 >> 4) + k * 2,
                 idesc_16<__nv_bfloat16>(128, C - k * 16, false), add || i != 0 || k != 0);
      }
    };

    for (int n = 0; n < n_chunk; ++n) {
      Stage &st = sm.st[n & 1];
      const Coef &cf = sm.c[n & 1];
      const uint32_t xq = me + TM_XQ + i0;
      const uint32_t par = n & 1u;
      bool bad = false;
      // the state's parts; the updates' of the chunk before, which they go over, have
      // been read with its outputs
      if (pending >= 0) wait_warp(&sm.o, pending & 1u);
      tc_fence_after();
      float top = 0.f, back_s = 1.f;  // back_s: S^T K^T to true numbers
      if (BF16) {
#pragma unroll
        for (int d = 0; d < SD; d += 16) {
          uint32_t x[8], y[8], z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) thirds(s[d + 2 * e], s[d + 2 * e + 1], x[e], y[e], z[e]);
          if (ok) {
            tmem_st8(me + TM_H + (d0 + d) / 2, x);
            tmem_st8(me + TM_H + 64 + (d0 + d) / 2, y);
            tmem_st8(me + TM_H + 128 + (d0 + d) / 2, z);
          }
        }
      } else {
#pragma unroll
        for (int d = 0; d < SD; d += 2) top = max_nan(top, s[d], s[d + 1]);
        top = of_both(0, top);
        const float up = power_for(top, 14, back_s);
#pragma unroll
        for (int d = 0; d < SD; d += 16) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) halves(s[d + 2 * e] * up, s[d + 2 * e + 1] * up, hi[e], lo[e]);
          if (ok) {
            tmem_st8(me + TM_H + (d0 + d) / 2, hi);
            tmem_st8(me + TM_H + 64 + (d0 + d) / 2, lo);
          }
        }
      }
      arrive(&sm.ps);
      wait_warp(&sm.full[n & 1], (n >> 1) & 1u);
      products(0, &sm.ps, par, [&]() {  // S^T K^T, then S^T Q^T
        const uint32_t kq = desc_lo(smem_u32(st.kq), 16);
#pragma unroll
        for (int k = 0; k < 8 * PARTS; ++k)
          if ((k & 7) < steps)
            mma_ts(tmem + TM_XK, tmem + TM_H + k * 8, kq + ((k & 7) >> 2) * (BLOCK >> 4) + (k & 3) * 2, id_t, k != 0);
        tc_commit(&sm.x);
      });
      put_outputs(true);
      // by another warp: issuing them takes as long as they run
      if (warp == 4) wait_warp(&sm.ps, par);
      products(4, &sm.pq, par, [&]() {
        const uint32_t kq = desc_lo(smem_u32(st.kq), 16);
#pragma unroll
        for (int k = 0; k < 8 * PARTS; ++k)
          if ((k & 7) < steps)
            mma_ts(tmem + TM_XQ, tmem + TM_H + k * 8, kq + (C * 128 >> 4) + ((k & 7) >> 2) * (BLOCK >> 4) + (k & 3) * 2, id_t, k != 0);
        tc_commit(&sm.xq);
      });
      // right sides
      wait_warp(&sm.x, par);
      tc_fence_after();
      float b[SC], x_top = 0.f;
#pragma unroll
      for (int part = 0; part < SC; part += 16) {
        uint32_t x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0u;
        if (ok) {
          tmem_ld16(me + TM_XK + i0 + part, x);
          tmem_wait_ld();
          tie16(x);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 f = cf.rhs[i0 + part + i];
          const float v = to_float<T>(st.v[(i0 + part + i) * LANES + l]);
          b[part + i] = fmaf(f.y, BF16 ? __uint_as_float(x[i]) : __uint_as_float(x[i]) * back_s, f.x * v);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) x_top = max_nan(x_top, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
      }
      top = 0.f;
#pragma unroll
      for (int i = 0; i < SC; i += 2) top = max_nan(top, b[i], b[i + 1]);
      // A column of the state that is not finite has nothing more to lose.
      bool lost = false;
      if (!(top <= MOST_SUM) || !(x_top * back_s <= MOST_SUM)) {
        float most = 0.f;
#pragma unroll
        for (int d = 0; d < SD; d += 2) most = max_nan(most, s[d], s[d + 1]);
        lost = !finite(most);
        bad = !lost;
      }
      wait_warp(&sm.xq, par);  // the state's parts have been read
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < SC; i += 16) {
        uint32_t x[8], y[8], z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) thirds(b[i + 2 * e], b[i + 2 * e + 1], x[e], y[e], z[e]);
        if (ok) {
          tmem_st8(me + TM_H + (i0 + i) / 2, x);
          tmem_st8(me + TM_H + 32 + (i0 + i) / 2, y);
          tmem_st8(me + TM_H + 64 + (i0 + i) / 2, z);
        }
      }
      arrive(&sm.pb);
      products(1, &sm.pb, par, [&]() {
        triangle(TM_XK, sm.t3, false);
        tc_commit(&sm.u);
      });
      // meanwhile the outputs' first part
      float most = 0.f;
      if (ok) {
#pragma unroll
        for (int part = 0; part < SC; part += 16) {
          uint32_t x[16];
          tmem_ld16(xq + part, x);
          tmem_wait_ld();
          tie16(x);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x[i] = __float_as_uint((BF16 ? __uint_as_float(x[i]) : __uint_as_float(x[i]) * back_s) * cf.eq[i0 + part + i]);
          tmem_st16(xq + part, x);
#pragma unroll
          for (int i = 0; i < 16; i += 2) most = max_nan(most, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
        }
      }
      // the updates
      wait_warp(&sm.u, par);
      if (ok) {
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < SC; part += 16) {
          uint32_t x[16];
          tmem_ld16(me + TM_XK + i0 + part, x);
          tmem_wait_ld();
          tie16(x);
#pragma unroll
          for (int i = 0; i < 16; ++i) b[part + i] = __uint_as_float(x[i]);
        }
      }
      float up_z = 1.f, back_z = 1.f;  // of what the state's step takes of them
      if (!BF16) {
        top = 0.f;
#pragma unroll
        for (int i = 0; i < SC; i += 2) {
          const float2 f = *reinterpret_cast<const float2 *>(&cf.until[i0 + i]);
          top = max_nan(top, b[i] * f.x, b[i + 1] * f.y);
        }
        top = of_both(1, top);
        up_z = power_for(top, 14, back_z);
      }
#pragma unroll
      for (int i = 0; i < SC; i += 16) {
        uint32_t x[8], y[8], z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = *reinterpret_cast<const float2 *>(&cf.until[i0 + i + 2 * e]);
          const float z0 = b[i + 2 * e] * f.x, z1 = b[i + 2 * e + 1] * f.y;
          if (BF16) {
            thirds(z0, z1, x[e], y[e], z[e]);
          } else {
            halves(z0 * up_z, z1 * up_z, x[e], y[e]);
          }
        }
        if (ok) {
          tmem_st8(me + TM_Z + (i0 + i) / 2, x);
          tmem_st8(me + TM_Z + 32 + (i0 + i) / 2, y);
          if (BF16) tmem_st8(me + TM_Z + 64 + (i0 + i) / 2, z);
        }
      }
      if (bad || (!lost && !finite(most))) *(volatile int *)&sm.chain_bad = n + 1;
      arrive(&sm.pz);
      products(2, &sm.pz, par, [&]() {
        const uint32_t kd = desc_lo(smem_u32(st.kq), BLOCK);
#pragma unroll
        for (int k = 0; k < 4 * PARTS; ++k) mma_ts(tmem + TM_S, tmem + TM_Z + k * 8, kd + (k & 3) * (2048 >> 4), id_kd, k != 0);
        tc_commit(&sm.s);
        tc_commit(&sm.empty[n & 1]);
      });
#pragma unroll
      for (int i = 0; i < SC; i += 16) {
        uint32_t x[8], y[8], z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) thirds(b[i + 2 * e], b[i + 2 * e + 1], x[e], y[e], z[e]);
        if (ok) {
          tmem_st8(me + TM_H + (i0 + i) / 2, x);
          tmem_st8(me + TM_H + 32 + (i0 + i) / 2, y);
          tmem_st8(me + TM_H + 64 + (i0 + i) / 2, z);
        }
      }
      const bool slow_prep = *(volatile int *)&sm.bad[n & 1] != 0;
      const float end = cf.end;
      arrive(&sm.py);
      products(3, &sm.py, par, [&]() {
        triangle(TM_XQ, st.p3, true);
        tc_commit(&sm.o);
        tc_commit(&sm.empty[n & 1]);  // with the state's step the last to read this stage
      });
      wait_warp(&sm.s, par);
      // one decision for all of the chain, whose threads meet at barriers on either way
      if (!any(slow_prep || *(volatile int *)&sm.chain_bad == n + 1)) {
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int part = 0; part < SD; part += 16) {
            uint32_t x[16];
            tmem_ld16(me + TM_S + d0 + part, x);
            tmem_wait_ld();
            tie16(x);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              s[part + i] = fmaf(s[part + i], end, BF16 ? __uint_as_float(x[i]) : __uint_as_float(x[i]) * back_z);
          }
          tc_fence_before();
        }
        pending = n;
        continue;
      }
      // The chunk row by row, from the inputs, as delta_rows.cu does it; the column's two
      // threads exchange their sums.
      wait_warp(&sm.o, par);  // its outputs are not wanted
      const int rows = min(C, nn - n * C);
#pragma unroll 1
      for (int i = 0; i < rows; ++i) {
        const int64_t tok = tok0 + n * C + i;
        const uint4 *kr = reinterpret_cast<const uint4 *>(p.k + tok * p.k_stride + hk * p.Dk);
        const uint4 *qr = reinterpret_cast<const uint4 *>(p.q + tok * p.q_stride + hk * p.Dk);
        float fk = 1.f, fq = 1.f, x[8], y[8];
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll 1
        for (int c = 0; c < p.Dk / 8; ++c) {
          unpack8<T>(__ldg(kr + c), x);
          unpack8<T>(__ldg(qr + c), y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            kk = fmaf(x[e], x[e], kk);
            qq = fmaf(y[e], y[e], qq);
          }
        }
        if (p.normalize) {
          fk = rsqrtf(kk + p.eps);
          fq = rsqrtf(qq + p.eps);
        }
#pragma unroll 1
        for (int c = 0; c < p.Dk / 8; ++c) {
          unpack8<T>(__ldg(kr + c), x);
          unpack8<T>(__ldg(qr + c), y);
#pragma unroll
          for (int e = 0; e < 8; ++e) kq = fmaf(x[e] * fk, y[e] * fq, kq);
        }
        float ks = 0.f, qs = 0.f;
#pragma unroll
        for (int c = 0; c < SD / 8; ++c)
          if (d0 + c * 8 < p.Dk) {
            unpack8<T>(__ldg(kr + d0 / 8 + c), x);
            unpack8<T>(__ldg(qr + d0 / 8 + c), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              ks = fmaf(x[e] * fk, s[c * 8 + e], ks);
              qs = fmaf(y[e] * fq, s[c * 8 + e], qs);
            }
          }
        sm.top[0][half][l] = ks;
        sm.top[1][half][l] = qs;
        named_sync(5 + (warp & 3), 64);
        ks = sm.top[0][0][l] + sm.top[0][1][l];
        qs = sm.top[1][0][l] + sm.top[1][1][l];
        named_sync(5 + (warp & 3), 64);
        const float decay = expf(__ldg(p.g + tok * p.Hv + h)), beta = __ldg(p.beta + tok * p.Hv + h);
        const float v = have ? to_float<T>(p.v[tok * p.v_stride + h * p.Dv + col]) : 0.f;
        const float u = beta * fmaf(-decay, ks, v);
#pragma unroll
        for (int c = 0; c < SD / 8; ++c)
          if (d0 + c * 8 < p.Dk) {
            unpack8<T>(__ldg(kr + d0 / 8 + c), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[c * 8 + e] = fmaf(x[e] * fk, u, decay * s[c * 8 + e]);
          }
        if (have && half == 0)
          p.out[(tok * p.Hv + h) * p.Dv + col] = (uint16_t)pack2<T>(p.scale * fmaf(kq, u, decay * qs), 0.f);
      }
    }
    put_outputs(false);
    if (ok && q.ok && q.dst >= 0 && have) {
      float *to = p.s + (((int64_t)q.dst * p.Hv + h) * p.Dk + d0) * p.Dv + col;
#pragma unroll
      for (int d = 0; d < SD; ++d)
        if (d0 + d < p.Dk) to[(int64_t)d * p.Dv] = s[d];
    }
  }
  // no product runs on when tensor memory is given back
  if (warp < 5 || warp == CHAIN / 32) {
    if (elect_one()) {
      tc_commit(&sm.drain);
      int never = 0;
      mbar_wait(&sm.drain, 0, &never);
    }
    __syncwarp();
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
    // the roles' exchange of registers waits for what a block is launched with
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, delta_chunk_kernel<T>)) != cudaSuccess) return e;
    if ((at.numRegs + 7) / 8 * 8 != LAUNCH_REGS) return cudaErrorInvalidConfiguration;
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
