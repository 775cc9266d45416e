// kvcache.cu -- what goes into the target's paged key-value cache, comes out
// of it and moves inside it (the target's pass over the tree: project page
// "Multi-Future Drafting", How it works, step 3, Figure 2 (c)).
//
//   append  norm of queries and keys per head, rotation, cache write
//           (optionally in E4M3 rows), in one pass over the packed projection
//   read    a stretch of positions back to a tensor
//   commit  the accepted path's entries to the context's end, in place
//
// All three move bytes: every element is read once and written once with
// 16-byte accesses (8-byte ones for the E4M3 form of 8 elements).  On the GPU
// alone (a captured call replayed):
//   append, 8 prompts of up to 2,000 tokens (15,500) of 16/4 heads of 256, fp16: 81
//     us, 4.7 TB/s, 0.70 of what a copy reaches; its issue slots are 78 % busy,
//     integer and shared-memory pipes next (50 %: addresses, factors, row sums)
//   append in E4M3 of 8 prompts of 512 such tokens, then the read of their
//     contexts of up to 12,000 positions in 16 bits: 476 MB in 99 us, 4.8 TB/s
//     (append 29 us, 3.1 TB/s; read 69 us, 5.6 TB/s, 0.82 of a copy)
//   commit: one block per request, a few kilobytes: its launch and three trips
//     to memory one after the other; 5.0 us for one request, 7.5 for 32
#include "kvcache.h"
#include "mfd_device.cuh"

namespace mfd {
namespace {

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_D = 256;
constexpr int UNROLL = 4;  // rows a lane of the read has in flight

// Page of position p of request q, or -1 (the caller reports).
__device__ __forceinline__ int page_of(const CacheView &c, int q, int64_t p) {
  const int64_t i = p >> c.ps_shift;
  if (p < 0 || i >= c.max_pages) return -1;
  const int g = __ldg(c.table + (size_t)q * c.max_pages + i);
  return g >= 0 && g < c.n_pages ? g : -1;
}

// ------------------------------------------------------------------ append

struct AppendParams {
  const uint8_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int T, N, Hq, Hk, D;
  const uint8_t *q_w, *k_w;
  float eps;
  const uint64_t *phase;
  int rot_dim, interleaved;
  const int32_t *pos, *ctx_len, *n_nodes;
  uint8_t *q_out, *k_out;
  CacheView cache;
  int32_t *status;
};

// cos and sin of 2 pi * (prod / 2^64): the quarter turn nearest to the angle
// is taken off in integers, so what is left keeps all of a float's bits.
__device__ __forceinline__ void turn_cos_sin(uint64_t prod, float &c, float &s) {
  const uint64_t quarter = (prod + (1ull << 61)) >> 62;
  const int64_t rest = (int64_t)(prod - (quarter << 62));  // [-2^61, 2^61)
  float s0, c0;
  sincospif((float)rest * 0x1p-63f, &s0, &c0);
  const int k = (int)(quarter & 3);
  c = k == 0 ? c0 : k == 1 ? -s0 : k == 2 ? -c0 : s0;
  s = k == 0 ? s0 : k == 1 ? c0 : k == 2 ? -s0 : -c0;
}

// Where the keys (and values) go.
enum { SINK_TENSOR = 0, SINK_CACHE = 1, SINK_E4M3 = 2 };

// One block handles up to WARPS * (32 / LR) * U rows (heads) of one token; a
// row of D elements is LR lanes of 8 elements (LR: the power of two at or above
// D / 8).  A block is short and waits for memory at its start: everything whose
// address is known (U rows a lane, weights, phases, lengths) is loaded before
// anything is used.
//
// Norm and rotation are one product of three: with r = 1 / sqrt(mean x^2 + eps),
//   y_e = r * (x_e (w_e cos a_e) + x_p (+- w_p sin a_e)),   p the partner of e,
// and the two bracketed factors are the same for every head of the token: the
// block makes them once, for queries and for keys, in shared memory.  A row is
// then one sum of squares and two products an element.  (With weights, cosines
// and sines applied one after the other the kernel waited for its own
// instructions: 16,000 tokens of 24 heads of 256 took 120 us.)
//
// Partners: another lane's chunk (halves of whole chunks: one shuffle of packed
// pairs), the lane's own pairs (interleaved), or, ROT_SMEM, two lanes' chunks at
// an offset; the row then passes through shared memory.
template <typename T, int SINK, int LR, int U, bool ROT_SMEM>
__global__ void __launch_bounds__(THREADS) append_kernel(const AppendParams p) {
  constexpr int RW = 32 / LR;  // rows of a warp at once
  pdl_launch_dependents();     // the attention that follows sets itself up meanwhile
  __shared__ float cos_s[MAX_D / 2], sin_s[MAX_D / 2];
  // w cos and +- w sin of queries and of keys, [half of a chunk][chunk]:
  // neighbouring lanes read neighbouring 16 bytes
  __shared__ float4 own_s[2][2][MAX_D / 8], other_s[2][2][MAX_D / 8];
  __shared__ float row_s[ROT_SMEM ? WARPS * RW : 1][ROT_SMEM ? MAX_D : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane & (LR - 1), sub = lane / LR;
  const int tok = blockIdx.x;
  const int q = tok / p.N, n = tok - q * p.N;
  const int rows = p.Hq + (SINK == SINK_TENSOR ? 1 : 2) * p.Hk;
  const bool in_row = c * 8 < p.D;
  const int row0 = (int)blockIdx.y * (WARPS * RW * U) + warp * RW + sub;

  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = row0 + u * WARPS * RW;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (in_row && row < rows) {  // before n_nodes is known: dead rows' values are not used
      const uint8_t *src;
      if (row < p.Hq)
        src = p.q + ((int64_t)tok * p.q_stride + row * p.D + c * 8) * 2;
      else if (row < p.Hq + p.Hk)
        src = p.k + ((int64_t)tok * p.k_stride + (row - p.Hq) * p.D + c * 8) * 2;
      else
        src = p.v + ((int64_t)tok * p.v_stride + (row - p.Hq - p.Hk) * p.D + c * 8) * 2;
      raw[u] = *reinterpret_cast<const uint4 *>(src);
    }
  }
  const int h = p.rot_dim >> 1;
  const bool turns = (int)threadIdx.x < h;  // h <= THREADS
  const uint64_t phase = turns ? __ldg(p.phase + threadIdx.x) : 0;
  const int64_t pos = turns ? __ldg(p.pos + tok) : 0;
  // this thread's two elements of the factors: weights of the element and its partner
  float w_own[2][2], w_other[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = threadIdx.x + i * THREADS;
    const int o = e >= 2 * h ? e : p.interleaved ? e ^ 1 : e < h ? e + h : e - h;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint8_t *w = k ? p.k_w : p.q_w;
      w_own[i][k] = w && e < p.D ? unpack2<T>(__ldg(reinterpret_cast<const uint16_t *>(w) + e)).x : 1.f;
      w_other[i][k] = w && e < p.D ? unpack2<T>(__ldg(reinterpret_cast<const uint16_t *>(w) + o)).x : 1.f;
    }
  }
  bool live = true;
  int ctx = 0, page = -1;
  if (SINK != SINK_TENSOR) {
    const int nn = p.n_nodes ? __ldg(p.n_nodes + q) : p.N;
    ctx = __ldg(p.ctx_len + q);
    const bool ok = nn >= 0 && nn <= p.N && ctx >= 0;
    if (!ok && threadIdx.x == 0) report(p.status, MFD_ERR_INPUT);
    live = ok && n < nn;
    if (live) page = page_of(p.cache, q, (int64_t)ctx + n);
    if (live && page < 0 && threadIdx.x == 0) report(p.status, MFD_ERR_INPUT);
  }
  if (turns) turn_cos_sin(phase * (uint64_t)pos, cos_s[threadIdx.x], sin_s[threadIdx.x]);
  block_sync();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = threadIdx.x + i * THREADS;
    if (e < p.D) {
      float cs = 1.f, sn = 0.f;
      if (e < 2 * h) {
        const bool second = p.interleaved ? (e & 1) : e >= h;
        const int a = p.interleaved ? e >> 1 : (second ? e - h : e);
        cs = cos_s[a];
        sn = second ? sin_s[a] : -sin_s[a];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        reinterpret_cast<float *>(&own_s[k][(e >> 2) & 1][e >> 3])[e & 3] = w_own[i][k] * cs;
        reinterpret_cast<float *>(&other_s[k][(e >> 2) & 1][e >> 3])[e & 3] = w_other[i][k] * sn;
      }
    }
  }
  block_sync();
  // the lane whose chunk holds this chunk's partners (halves of whole chunks)
  const int hc = h >> 3;
  const int partner = c < hc ? lane + hc : c < 2 * hc ? lane - hc : lane;
  const bool paired = c < 2 * hc;
  const float per_d = 1.f / (float)p.D;
  // the token's place in the cache, in elements
  const int slot = (ctx + n) & ((1 << p.cache.ps_shift) - 1);
  const int64_t place = SINK == SINK_TENSOR ? 0 : page * p.cache.page_stride + slot * p.cache.token_stride + c * 8;

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = row0 + u * WARPS * RW;
    if (row0 - sub + u * WARPS * RW >= rows) break;  // the same for the whole warp
    const bool have = row < rows;
    const bool is_q = row < p.Hq, is_v = row >= p.Hq + p.Hk;
    float x[8];
    unpack8<T>(raw[u], x);
    if (!__all_sync(0xffffffffu, is_v)) {
      // partners, from the values as they came
      float xp[8];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) xp[i] = c * 8 + i < 2 * h ? x[i ^ 1] : 0.f;
      } else if (ROT_SMEM) {
        float *buf = row_s[warp * RW + sub];
        __syncwarp();
        if (in_row)
#pragma unroll
          for (int i = 0; i < 8; ++i) buf[c * 8 + i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = c * 8 + i;
          xp[i] = e < 2 * h ? buf[e < h ? e + h : e - h] : 0.f;
        }
      } else {
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, raw[u].x, partner);
        o.y = __shfl_sync(0xffffffffu, raw[u].y, partner);
        o.z = __shfl_sync(0xffffffffu, raw[u].z, partner);
        o.w = __shfl_sync(0xffffffffu, raw[u].w, partner);
        if (!paired) o = make_uint4(0, 0, 0, 0);
        unpack8<T>(o, xp);
      }
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = 1; o < LR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!is_v && in_row) {
        const float r = (is_q ? p.q_w : p.k_w) ? rsqrtf(fmaf(ss, per_d, p.eps)) : 1.f;
        const int k = is_q ? 0 : 1;
        const float4 a = own_s[k][0][c], b = own_s[k][1][c], d = other_s[k][0][c], e = other_s[k][1][c];
        x[0] = r * fmaf(xp[0], d.x, x[0] * a.x);
        x[1] = r * fmaf(xp[1], d.y, x[1] * a.y);
        x[2] = r * fmaf(xp[2], d.z, x[2] * a.z);
        x[3] = r * fmaf(xp[3], d.w, x[3] * a.w);
        x[4] = r * fmaf(xp[4], e.x, x[4] * b.x);
        x[5] = r * fmaf(xp[5], e.y, x[5] * b.y);
        x[6] = r * fmaf(xp[6], e.z, x[6] * b.z);
        x[7] = r * fmaf(xp[7], e.w, x[7] * b.w);
      }
    }
    // out
    if (is_q || SINK == SINK_TENSOR) {
      if (have && in_row) {
        uint8_t *dst = is_q ? p.q_out + (((int64_t)tok * p.Hq + row) * p.D + c * 8) * 2
                            : p.k_out + (((int64_t)tok * p.Hk + row - p.Hq) * p.D + c * 8) * 2;
        *reinterpret_cast<uint4 *>(dst) = live ? pack8<T>(x) : make_uint4(0, 0, 0, 0);
      }
    } else if (SINK == SINK_CACHE) {
      if (have && in_row && page >= 0) {
        const int hd = row - p.Hq - (is_v ? p.Hk : 0);
        uint8_t *dst = static_cast<uint8_t *>(is_v ? p.cache.v : p.cache.k) + (place + hd * p.cache.head_stride) * 2;
        *reinterpret_cast<uint4 *>(dst) = is_v ? raw[u] : pack8<T>(x);
      }
    }
    if (SINK == SINK_E4M3) {
      // the row's largest magnitude (the shuffles take the whole warp)
      uint32_t am = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
      for (int o = 1; o < LR; o <<= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
      if (!is_q && have && in_row && page >= 0) {
        const int code = e4m3_code(am);
        uint2 b = make_uint2(0, 0);
        if (code != EXP_NAN) {
          const float inv = e4m3_inv(code), lim = e4m3_limit<T>(code);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= inv;
          if (lim < 448.f)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -lim), lim);
          b.x = e4m3x4(x[0], x[1], x[2], x[3]);
          b.y = e4m3x4(x[4], x[5], x[6], x[7]);
        }
        const int hd = row - p.Hq - (is_v ? p.Hk : 0);
        uint8_t *dst = static_cast<uint8_t *>(is_v ? p.cache.v : p.cache.k) + place + hd * p.cache.head_stride;
        *reinterpret_cast<uint2 *>(dst) = b;
        if (c == 0)
          (is_v ? p.cache.v_exp : p.cache.k_exp)[(((int64_t)page * p.Hk + hd) << p.cache.ps_shift) + slot] =
              (uint8_t)code;
      }
    }
  }
}

template <typename T, int SINK, int LR, int U>
cudaError_t launch_append_u(const AppendParams &p, int rows, cudaStream_t stream) {
  const int per = WARPS * (32 / LR) * U;
  const dim3 grid(p.T, (rows + per - 1) / per);
  if (!p.interleaved && (p.rot_dim / 2) % 8 != 0)
    append_kernel<T, SINK, LR, U, true><<<grid, THREADS, 0, stream>>>(p);
  else
    append_kernel<T, SINK, LR, U, false><<<grid, THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

// Rows a lane: as many as one block needs for a token, up to 6.
template <typename T, int SINK, int LR>
cudaError_t launch_append_lr(const AppendParams &p, cudaStream_t stream) {
  const int rows = p.Hq + (SINK == SINK_TENSOR ? 1 : 2) * p.Hk;
  const int need = (rows + WARPS * (32 / LR) - 1) / (WARPS * (32 / LR));
  return need <= 3 ? launch_append_u<T, SINK, LR, 3>(p, rows, stream) : launch_append_u<T, SINK, LR, 6>(p, rows, stream);
}

template <typename T, int SINK>
cudaError_t launch_append_sink(const AppendParams &p, cudaStream_t stream) {
  if (p.D <= 64) return launch_append_lr<T, SINK, 8>(p, stream);
  if (p.D <= 128) return launch_append_lr<T, SINK, 16>(p, stream);
  return launch_append_lr<T, SINK, 32>(p, stream);
}

template <typename T>
cudaError_t launch_append_t(const AppendParams &p, int sink, cudaStream_t stream) {
  switch (sink) {
    case SINK_TENSOR: return launch_append_sink<T, SINK_TENSOR>(p, stream);
    case SINK_CACHE: return launch_append_sink<T, SINK_CACHE>(p, stream);
    default: return launch_append_sink<T, SINK_E4M3>(p, stream);
  }
}

// -------------------------------------------------------------------- read

// One lane moves 16 bytes of the cache (8 elements, or 16 E4M3 ones); a row of
// D is LR lanes of that; a block moves WARPS * (32 / LR) * UNROLL rows
// (position, head) of one request, keys (blockIdx.z = 0) or values.
template <typename T, bool E4M3, int LR>
__global__ void __launch_bounds__(THREADS)
    read_kernel(const CacheView cv, int L_max, const int32_t *__restrict__ start, const int32_t *__restrict__ length,
                uint8_t *k_out, uint8_t *v_out, int32_t *status) {
  constexpr int RW = 32 / LR, EL = E4M3 ? 16 : 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane & (LR - 1), sub = lane / LR;
  const int q = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  if (c * EL >= cv.D) return;
  const int st = __ldg(start + q), len = __ldg(length + q);
  const bool ok = st >= 0 && len >= 0 && len <= L_max;
  if (!ok && threadIdx.x == 0) report(status, MFD_ERR_INPUT);
  const int64_t rows = (int64_t)L_max * cv.Hk;
  const int64_t row0 = (int64_t)blockIdx.x * (WARPS * RW * UNROLL) + warp * RW + sub;
  const uint8_t *base = static_cast<const uint8_t *>(is_v ? cv.v : cv.k);
  const uint8_t *exps = is_v ? cv.v_exp : cv.k_exp;
  uint4 raw[UNROLL];
  int code[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int64_t row = row0 + u * WARPS * RW;
    raw[u] = make_uint4(0, 0, 0, 0);
    code[u] = 0;
    if (row < rows && ok) {
      int i, hd;  // position and head
      if (rows < (1ll << 31)) {
        i = (int)((uint32_t)row / (uint32_t)cv.Hk);
        hd = (int)row - i * cv.Hk;
      } else {
        i = (int)(row / cv.Hk);
        hd = (int)(row - (int64_t)i * cv.Hk);
      }
      if (i < len) {
        const int64_t pos = (int64_t)st + i;
        const int page = page_of(cv, q, pos);
        if (page < 0) {
          report(status, MFD_ERR_INPUT);
        } else {
          const int slot = (int)(pos & ((1 << cv.ps_shift) - 1));
          const int64_t e = page * cv.page_stride + hd * cv.head_stride + slot * cv.token_stride + c * EL;
          raw[u] = *reinterpret_cast<const uint4 *>(base + e * (E4M3 ? 1 : 2));
          if (E4M3) code[u] = exps[(((int64_t)page * cv.Hk + hd) << cv.ps_shift) + slot];
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int64_t row = row0 + u * WARPS * RW;
    if (row >= rows) break;
    uint4 *dst = reinterpret_cast<uint4 *>((is_v ? v_out : k_out) + (((int64_t)q * rows + row) * cv.D + c * EL) * 2);
    if (E4M3) {
      const float s = e4m3_scale(code[u]);
      const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = e4m3x2_float(w[i >> 1] >> (16 * (i & 1)) & 0xFFFFu);
        o[i] = pack2<T>(f.x * s, f.y * s);
      }
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
      *dst = raw[u];
    }
  }
}

template <typename T, bool E4M3>
cudaError_t launch_read_t(const KvReadLaunch &A, cudaStream_t stream) {
  const int lanes = A.cache.D / (E4M3 ? 16 : 8);
  const int LR = lanes <= 4 ? 4 : lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
  const int64_t per = WARPS * (32 / LR) * UNROLL;
  const dim3 grid((unsigned)(((int64_t)A.L_max * A.cache.Hk + per - 1) / per), A.n_req, 2);
  uint8_t *ko = static_cast<uint8_t *>(A.k_out), *vo = static_cast<uint8_t *>(A.v_out);
  switch (LR) {
    case 4: read_kernel<T, E4M3, 4><<<grid, THREADS, 0, stream>>>(A.cache, A.L_max, A.start, A.length, ko, vo, A.status); break;
    case 8: read_kernel<T, E4M3, 8><<<grid, THREADS, 0, stream>>>(A.cache, A.L_max, A.start, A.length, ko, vo, A.status); break;
    case 16: read_kernel<T, E4M3, 16><<<grid, THREADS, 0, stream>>>(A.cache, A.L_max, A.start, A.length, ko, vo, A.status); break;
    default: read_kernel<T, E4M3, 32><<<grid, THREADS, 0, stream>>>(A.cache, A.L_max, A.start, A.length, ko, vo, A.status); break;
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------------ commit

constexpr int MAX_L = 16;
constexpr int COMMIT_THREADS = 512;

// One block per request, one warp per (head, keys or values) at a time.  The
// path increases, so path[j] >= j: an entry's new place may be another entry's
// old one, and every entry is read before any is written.
__global__ void __launch_bounds__(COMMIT_THREADS)
    commit_kernel(const CacheView cv, int L, const int32_t *ctx_len, const int32_t *__restrict__ accept_len,
                  const int32_t *__restrict__ path, const int32_t *__restrict__ n_nodes, int32_t *new_len,
                  int32_t *status) {
  const int q = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctx = ctx_len[q], acc = __ldg(accept_len + q), nn = __ldg(n_nodes + q);
  // lane j checks step j and finds its entries' places
  int src_page = -1, dst_page = -1;
  const int node = lane <= L ? __ldg(path + (size_t)q * (L + 1) + lane) : 0;
  const int up = __shfl_up_sync(0xffffffffu, node, 1);
  bool ok = ctx >= 0 && acc >= 0 && acc <= L;
  if (ok && lane <= acc) {
    const int before = lane ? up : -1;
    src_page = page_of(cv, q, (int64_t)ctx + node);
    dst_page = page_of(cv, q, (int64_t)ctx + lane);
    ok = node > before && node < nn && (lane > 0 || node == 0) && src_page >= 0 && dst_page >= 0;
  }
  ok = __all_sync(0xffffffffu, ok);
  block_sync();  // new_len may be ctx_len: every warp has read it
  if (threadIdx.x == 0) {
    new_len[q] = ok ? ctx + acc + 1 : ctx;
    if (!ok) report(status, MFD_ERR_INPUT);
  }
  if (!ok) return;
  const int esz = cv.dtype == MFD_E4M3 ? 1 : 2;
  const int chunks = cv.D * esz / 16;  // 1..32
  const int mask = (1 << cv.ps_shift) - 1;
  for (int w = warp; w < 2 * cv.Hk; w += COMMIT_THREADS / 32) {
    const int hd = w >> 1;
    uint8_t *base = static_cast<uint8_t *>((w & 1) ? cv.v : cv.k) + hd * cv.head_stride * esz + lane * 16;
    uint8_t *exps = (w & 1) ? cv.v_exp : cv.k_exp;
    uint4 e[MAX_L];
#pragma unroll
    for (int j = 1; j <= MAX_L; ++j) {
      const int pg = __shfl_sync(0xffffffffu, src_page, j), nd = __shfl_sync(0xffffffffu, node, j);
      if (j <= acc && lane < chunks)
        e[j - 1] = *reinterpret_cast<const uint4 *>(base + (pg * cv.page_stride + ((ctx + nd) & mask) * cv.token_stride) * esz);
    }
    uint8_t code = 0;
    if (exps && lane >= 1 && lane <= acc)
      code = exps[(((int64_t)src_page * cv.Hk + hd) << cv.ps_shift) + ((ctx + node) & mask)];
    __syncwarp();
#pragma unroll
    for (int j = 1; j <= MAX_L; ++j) {
      const int pg = __shfl_sync(0xffffffffu, dst_page, j);
      if (j <= acc && lane < chunks)
        *reinterpret_cast<uint4 *>(base + (pg * cv.page_stride + ((ctx + j) & mask) * cv.token_stride) * esz) = e[j - 1];
    }
    if (exps && lane >= 1 && lane <= acc)
      exps[(((int64_t)dst_page * cv.Hk + hd) << cv.ps_shift) + ((ctx + lane) & mask)] = code;
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendLaunch &A, cudaStream_t stream) {
  AppendParams p;
  p.q = static_cast<const uint8_t *>(A.q);
  p.k = static_cast<const uint8_t *>(A.k);
  p.v = static_cast<const uint8_t *>(A.v);
  p.q_stride = A.q_stride;
  p.k_stride = A.k_stride;
  p.v_stride = A.v_stride;
  p.T = A.n_req * A.N;
  p.N = A.N;
  p.Hq = A.Hq;
  p.Hk = A.Hk;
  p.D = A.D;
  p.q_w = static_cast<const uint8_t *>(A.q_w);
  p.k_w = static_cast<const uint8_t *>(A.k_w);
  p.eps = A.eps;
  p.phase = A.phase;
  p.rot_dim = A.rot_dim;
  p.interleaved = A.interleaved;
  p.pos = A.pos;
  p.ctx_len = A.ctx_len;
  p.n_nodes = A.n_nodes;
  p.q_out = static_cast<uint8_t *>(A.q_out);
  p.k_out = static_cast<uint8_t *>(A.k_out);
  p.status = A.status;
  int sink = SINK_TENSOR;
  if (A.cache) {
    p.cache = *A.cache;
    sink = A.cache->dtype == MFD_E4M3 ? SINK_E4M3 : SINK_CACHE;
  } else {
    p.cache = CacheView{};
  }
  return A.dtype == MFD_BF16 ? launch_append_t<__nv_bfloat16>(p, sink, stream)
                             : launch_append_t<__half>(p, sink, stream);
}

cudaError_t launch_kv_read(const KvReadLaunch &A, cudaStream_t stream) {
  if (A.cache.dtype == MFD_E4M3)
    return A.dtype == MFD_BF16 ? launch_read_t<__nv_bfloat16, true>(A, stream) : launch_read_t<__half, true>(A, stream);
  return launch_read_t<__nv_bfloat16, false>(A, stream);  // 16-bit entries are copied as they are
}

cudaError_t launch_kv_commit(const KvCommitLaunch &A, cudaStream_t stream) {
  commit_kernel<<<A.n_req, COMMIT_THREADS, 0, stream>>>(A.cache, A.L, A.ctx_len, A.accept_len, A.path, A.n_nodes,
                                                        A.new_len, A.status);
  return cudaGetLastError();
}

}  // namespace mfd
