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
// other: a block's warps share the rows' vectors.  A block walks (request, head,
// slice) items.  While it works on one, the next one's path is read, then its
// rows' vectors go to shared memory and its state to L2, so that only the state's
// way from there is waited for.
//
// One token reads and writes the state once: 64 requests of 32 heads of 128 x 128
// take 49 us, 5.5 TB/s of the states' 268 MB.  A path reads it once as well, but
// its rows follow one another, each for as long as its exchanges take: 32 paths of up to
// 16 rows take 38 us, of which the states' bytes are 18.
#include "delta.h"
#include "kvcache.h"
#include "mfd_device.cuh"

namespace mfd {
namespace {

constexpr int COLS = 16;     // of a warp
constexpr int BATCH = DELTA_MAX_DEPTH + 1;  // rows at most: all of a path
static_assert(BATCH >= DELTA_CHUNK_FROM - 1, "rows of the rule");
constexpr int MAX_DK = 128;
constexpr int PER = MAX_DK / 8;  // rows of the state a lane holds
constexpr int ORDERED = 256;     // requests at most that a block puts in order

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

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <typename T, int WARPS, int MODE>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) delta_rows_kernel(const DeltaArgs p, int slices, int items) {
  constexpr int W = WARPS * COLS, THREADS = WARPS * 32, VECS = MODE == COMMIT ? 1 : 2;
  __shared__ float4 k_s[BATCH][MAX_DK / 4], q_s[MODE == COMMIT ? 1 : BATCH][MAX_DK / 4];
  __shared__ uint4 raw_s[2][BATCH][VECS][MAX_DK / 8], v_s[2][BATCH][W / 8];  // as they are, of this item and the next
  __shared__ float g_s[2][BATCH], b_s[2][BATCH], decay_s[BATCH], beta_s[BATCH], qk_s[BATCH];
  __shared__ int row_s[2][BATCH], bad_s[2], length_s[ORDERED], order_s[ORDERED];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = lane >> 2, per = p.Dk / 8;  // rows of a group
  pdl_launch_dependents();
  pdl_wait();
  if (tid < 2) bad_s[tid] = 0;
  if (per < PER) {  // narrower keys leave elements between the groups': zeros, like the state's rows there
    for (int i = tid; i < BATCH * MAX_DK; i += THREADS) reinterpret_cast<float *>(k_s)[i] = 0.f;
    for (int i = tid; i < (MODE == COMMIT ? 1 : BATCH) * MAX_DK; i += THREADS) reinterpret_cast<float *>(q_s)[i] = 0.f;
  }
  // Blocks that walk several items get them longest first, and every second round in
  // reverse: their sums of rows differ by little then.
  const bool ordered = (int)gridDim.x < items && p.n_req <= ORDERED && (MODE == COMMIT || (p.n_nodes && p.N > 1));
  if (ordered) {
    for (int i = tid; i < p.n_req; i += THREADS) length_s[i] = __ldg((MODE == COMMIT ? p.accept_len : p.n_nodes) + i);
    block_sync();
    for (int i = tid; i < p.n_req; i += THREADS) {
      const int own = length_s[i];
      int place = 0;
      for (int j = 0; j < p.n_req; ++j) place += length_s[j] > own || (length_s[j] == own && j < i);
      order_s[place] = i;
    }
    block_sync();
  }
  auto item_of = [&](int round) { return round * (int)gridDim.x + (int)(round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); };
  struct Item {
    int slice, h, r, nn, src, dst, rows;
    int node;  // of the path, thread's
  };
  // What a request says of itself, not looked at yet.
  auto read = [&](int item) {
    Item x;
    x.slice = item % slices;
    x.h = item / slices % p.Hv;
    x.r = item / slices / p.Hv;
    if (ordered) x.r = order_s[x.r];
    x.nn = p.n_nodes ? __ldg(p.n_nodes + x.r) : p.N;
    x.src = p.src ? __ldg(p.src + x.r) : x.r;
    x.dst = p.dst ? __ldg(p.dst + x.r) : x.src;
    x.rows = MODE == COMMIT ? __ldg(p.accept_len + x.r) : 0;
    x.node = MODE == COMMIT && tid <= p.L ? __ldg(p.path + (int64_t)x.r * (p.L + 1) + tid) : 0;
    return x;
  };
  // Looks at it, by all threads: false where numbers are wrong; the path's nodes are
  // judged by their threads, and known after a barrier.
  auto check = [&](Item &x, int buf) {
    const bool ok = x.nn >= 0 && x.nn <= p.N && x.src >= -1 && x.src < p.n_slots && x.dst >= -1 && x.dst < p.n_slots &&
                    (MODE == RULE || (x.rows >= 0 && x.rows <= p.L));
    x.rows = !ok ? -1 : MODE == COMMIT ? x.rows + 1 : x.nn;
    if (MODE == COMMIT && tid < 32) {
      const int before = __shfl_up_sync(0xffffffffu, x.node, 1);
      if (tid < x.rows) {
        if (x.node >= x.nn || (tid == 0 ? x.node != 0 : x.node <= before)) bad_s[buf] = 1;
        row_s[buf][tid] = x.node;
      }
    }
  };
  // Its rows' vectors on their way to buffer `buf`, its state's to L2.
  auto fetch = [&](const Item &x, int buf, bool state) {
    const int hk = x.h / (p.Hv / p.Hk), n = x.rows, at0 = x.slice * W;
    const int64_t tok0 = (int64_t)x.r * p.N;
    auto token = [&](int i) { return tok0 + (MODE == COMMIT ? row_s[buf][i] : i); };
    for (int i = tid; i < n * VECS * (MAX_DK / 8); i += THREADS) {
      const int c = i % (MAX_DK / 8), vec = i / (MAX_DK / 8) % VECS, row = i / (MAX_DK / 8) / VECS;
      if (c * 8 < p.Dk)
        cp_async16(&raw_s[buf][row][vec][c], (vec ? p.q + token(row) * p.q_stride : p.k + token(row) * p.k_stride) + hk * p.Dk + c * 8);
    }
    for (int i = tid; i < n * (W / 8); i += THREADS) {
      const int row = i / (W / 8), c = i % (W / 8);
      if (at0 + c * 8 < p.Dv) cp_async16(&v_s[buf][row][c], p.v + token(row) * p.v_stride + x.h * p.Dv + at0 + c * 8);
    }
    if (tid < n) {
      cp_async4(&g_s[buf][tid], p.g + token(tid) * p.Hv + x.h);
      cp_async4(&b_s[buf][tid], p.beta + token(tid) * p.Hv + x.h);
    }
    if (state && x.src >= 0)
      for (int i = tid; i < p.Dk; i += THREADS)
        bulk_prefetch_l2(p.s + (((int64_t)x.src * p.Hv + x.h) * p.Dk + i) * p.Dv + at0, (uint32_t)min(W, p.Dv - at0) * 4);
  };

  int buf = 0;
  Item x = read(blockIdx.x);
  block_sync();
  check(x, 0);
  block_sync();
  if (bad_s[0]) x.rows = -1;
  if (x.rows > 0) fetch(x, 0, false);
  for (int round = 0, item = blockIdx.x; item < items; buf ^= 1) {
    const int n = max(x.rows, 0), h = x.h, slice = x.slice;
    const int col = slice * W + warp * COLS + (lane & 3) * 4;
    const bool have = col < p.Dv;
    const int64_t tok0 = (int64_t)x.r * p.N;
    float4 S[PER];
    {
      const float *from = p.s + (((int64_t)x.src * p.Hv + h) * p.Dk + group * per) * p.Dv + col;
#pragma unroll
      for (int t = 0; t < PER; ++t)
        S[t] = x.rows >= 0 && x.src >= 0 && have && t < per ? *reinterpret_cast<const float4 *>(from + (int64_t)t * p.Dv)
                                                            : make_float4(0, 0, 0, 0);
    }
    const int next = item_of(++round);
    Item y = x;
    if (next < items) y = read(next);
    if (x.rows < 0 && tid == 0) report(p.status, MFD_ERR_INPUT);
    // rows that are not live
    if (MODE == RULE && have)
      for (int i = n + group; i < p.N; i += 8)
        *reinterpret_cast<uint2 *>(p.out + ((tok0 + i) * p.Hv + h) * p.Dv + col) = make_uint2(0, 0);
    asm volatile("cp.async.wait_all;" ::: "memory");
    block_sync();
    // half a warp for a key, half for a query
    for (int i = warp; i < n; i += WARPS) {
      const int c = lane & 15, vec = lane >> 4;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (c * 8 < p.Dk && vec < VECS) raw = raw_s[buf][i][vec & (VECS - 1)][c];
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
      if (vec < VECS) {
        // element e of the vector is element e % per of group e / per; rows of groups are
        // PER floats apart in shared memory, whatever Dk is
        float *to = reinterpret_cast<float *>(vec ? q_s[MODE == COMMIT ? 0 : i] : k_s[i]);
        if (per == PER) {
          *reinterpret_cast<float4 *>(to + c * 8) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4 *>(to + c * 8 + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int at = c * 8 + e;
            if (at < p.Dk) *reinterpret_cast<float2 *>(to + at / per * PER + at % per) = make_float2(x[e], x[e + 1]);
          }
        }
      }
      if (lane == 0) {
        decay_s[i] = expf(g_s[buf][i]);
        beta_s[i] = b_s[buf][i];
        qk_s[i] = qk;
      }
    }
    if (tid == 0) bad_s[buf] = 0;  // looked at; the next but one's
    if (next < items) check(y, buf ^ 1);
    block_sync();
    if (next < items) {
      if (bad_s[buf ^ 1]) y.rows = -1;
      if (y.rows > 0) fetch(y, buf ^ 1, true);
    }

    // The state is S times `kept`, the product of the decays since it was last multiplied
    // out: a row then costs two products an element, not three.
    float kept = 1.f;
    for (int i = 0; i < n; ++i) {
      const uint2 raw = reinterpret_cast<const uint2 *>(v_s[buf][i])[warp * (COLS / 4) + (lane & 3)];
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
      // A decay too small to divide by, or NaN; or a step that divided by it would leave
      // fp32 (the state itself, undivided, holds it).  A column's lanes have the same sums.
      const float most = fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(u.z), fabsf(u.w)));
      if (!(d > 0x1p-40f && d < 0x1p40f) || most > d * 0x1p100f) {
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
        *reinterpret_cast<uint2 *>(p.out + ((tok0 + i) * p.Hv + h) * p.Dv + col) =
            make_uint2(pack2<T>(p.scale * fmaf(qk, u.x, d * b.x), p.scale * fmaf(qk, u.y, d * b.y)),
                       pack2<T>(p.scale * fmaf(qk, u.z, d * b.z), p.scale * fmaf(qk, u.w, d * b.w)));
      }
    }
    if (x.rows >= 0 && x.dst >= 0 && have) {
      float *to = p.s + (((int64_t)x.dst * p.Hv + h) * p.Dk + group * per) * p.Dv + col;
#pragma unroll
      for (int t = 0; t < PER; ++t)
        if (t < per)
          *reinterpret_cast<float4 *>(to + (int64_t)t * p.Dv) = make_float4(kept * S[t].x, kept * S[t].y, kept * S[t].z, kept * S[t].w);
    }
    x = y;
    item = next;
  }
}

template <typename T, int WARPS, int MODE>
cudaError_t launch_width(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  const int slices = (A.Dv + WARPS * COLS - 1) / (WARPS * COLS);
  const int64_t items = (int64_t)A.n_req * A.Hv * slices, resident = (int64_t)n_sm * (16 / WARPS);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(items < resident ? items : resident));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = stream;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, delta_rows_kernel<T, WARPS, MODE>, A, slices, (int)items);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int MODE>
cudaError_t launch_mode(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  // Narrower slices where few heads leave SMs without work, for one token: of 4 requests of
  // 32 heads it takes 5.9 us so, 6.6 with four warps; of 8 requests 9.1 and 7.4.  Blocks
  // that have rows to do in turn, or a path, are no faster so: 6.0 and 5.6 us for one
  // request's path; 17 rows of one request 21.1 and 19.1 us, of 4 requests 23.2 and 21.1
  // (a call by events, the L2 cache flushed before it).
  const int64_t heads = (int64_t)A.n_req * A.Hv;
  if (MODE == RULE && A.N == 1 && heads * ((A.Dv + 63) / 64) <= 2 * n_sm) return launch_width<T, 2, RULE>(A, n_sm, stream);
  return launch_width<T, 4, MODE>(A, n_sm, stream);
}
template <int MODE>
cudaError_t launch_type(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  return A.dtype == MFD_BF16 ? launch_mode<__nv_bfloat16, MODE>(A, n_sm, stream) : launch_mode<__half, MODE>(A, n_sm, stream);
}

}  // namespace

cudaError_t launch_delta_rows(const DeltaArgs &A, int n_sm, cudaStream_t stream) { return launch_type<RULE>(A, n_sm, stream); }
cudaError_t launch_delta_commit(const DeltaArgs &A, int n_sm, cudaStream_t stream) { return launch_type<COMMIT>(A, n_sm, stream); }

}  // namespace mfd
