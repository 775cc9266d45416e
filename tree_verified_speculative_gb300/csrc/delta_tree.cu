// delta_tree.cu -- the gated delta rule over a tree's nodes, each behind its own
// path, from a state that stays (the method's pages name tree kernels for hybrid
// targets: model card "MFD drafter for Qwen3.5-4B", Usage).
//
// Unrolled along a path, a node's update and output are sums over the nodes
// above it, at most 16.  The root is done first, into the state that all others
// start from; for a node i below it, with c the sum of g along its path and r, s
// the factors that the norms give its key and query,
//
//   u_i = beta_i (v_i - e^(c_i) r_i S^T k_i)
//         - sum_{j above i} beta_i r_i r_j e^(c_i - c_j) (k_i . k_j) u_j
//   o_i = scale s_i (e^(c_i) S^T q_i + sum_{j above i, or i} r_j e^(c_i - c_j) (q_i . k_j) u_j)
//
// The products with the state, and of queries and keys with keys, are 64 nodes
// at a time on the tensor cores; the sums run level by level of the tree, a node
// a warp, over the nodes above it alone, so that what a node holds reaches no
// node beside it.  Nodes are sorted by depth.
//
// Keys and queries go to the tensor cores as they are.  The state goes in as a
// sum of numbers of their type: three of bf16, each the front of what is left
// (24 bits), or two of fp16 after a power of two for each column (22 bits).
#include <atomic>
#include <type_traits>

#include "delta_tc.cuh"

namespace mfd {
namespace {

constexpr int C = 64;        // nodes of a block
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int DEPTH = DELTA_MAX_DEPTH;
constexpr int MAX_DK = 128;
constexpr int HALF = 128 * 128;  // 64 columns of a block's keys and queries
constexpr int DS = DEPTH + 1;    // floats of a row of the dot products' table

// Tensor memory, columns.
constexpr int TM_S = 0;    // the state's parts, 64 each
constexpr int TM_X = 192;  // S^T [K; Q]^T
constexpr int TM_G = 320;  // [K; Q] K'^T of two blocks

struct Node {
  float chi, clo, beta, rk, rq;
  int at;  // node, and its depth from bit 16
};
struct Entry {  // what a sum over the nodes above takes of one
  float a, b;
  int at, pad;
};
struct Fixed {
  uint64_t mma, drain;
  uint32_t tmem;
  int bad, abort;
  float root[4];  // decay, beta, q . k
  int level[DEPTH + 2];
  int hist[DEPTH + 1][32], count[DEPTH + 1];
  float k0[MAX_DK], q0[MAX_DK];
};
// The rest of shared memory, by the number of nodes.
struct Layout {
  int kc, dots, entries, u, node, above, par, depth, pos, fixed, total;
};
__host__ __device__ inline Layout layout(int N, int lanes) {
  const int n = N > 1 ? N - 1 : 1;
  Layout y;
  int at = 2 * HALF;  // keys' 64 rows, then queries', later S^T Q^T
  y.kc = at;          // another block's keys, later the values
  at += C * 256;
  y.dots = at;
  at += 2 * C * DS * 4;
  // the nodes' entries, and before that the rows of nodes above as bits; where a
  // block has 64 columns S^T Q^T leaves them room
  y.entries = lanes == 64 ? HALF : at;
  at += lanes == 64 ? 0 : C * DEPTH * (int)sizeof(Entry);
  y.u = at;
  at += n * lanes * 4;
  y.node = at;
  at += n * (int)sizeof(Node);
  y.above = at;
  at += n * DEPTH * 2;
  y.par = at;
  at += (N * 2 + 15) / 16 * 16;
  y.pos = at;
  at += (N * 2 + 15) / 16 * 16;
  y.depth = at;
  at += (N + 15) / 16 * 16;
  y.fixed = (at + 15) / 16 * 16;
  y.total = y.fixed + (int)sizeof(Fixed);
  return y;
}

// Columns of a state in a block: as many as fit with all nodes' updates.
inline int lanes_for(int N) { return N <= 257 ? 128 : 64; }

template <typename T, int LN>  // LN: columns a lane has in the sums
__global__ void __launch_bounds__(THREADS, 1) delta_tree_kernel(const DeltaArgs p, int slices) {
  constexpr int LANES = 32 * LN;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int PARTS = BF16 ? 3 : 2;
  constexpr int ISSUER = WARPS - 1;  // the warp that starts products
  extern __shared__ uint8_t raw_smem[];
  uint8_t *sm = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  const Layout y = layout(p.N, LANES);
  Fixed &fx = *reinterpret_cast<Fixed *>(sm + y.fixed);
  uint8_t *tile = sm, *kc = sm + y.kc;
  float *xq = reinterpret_cast<float *>(sm), *dots = reinterpret_cast<float *>(sm + y.dots), *u_s = reinterpret_cast<float *>(sm + y.u);
  uint16_t *v_s = reinterpret_cast<uint16_t *>(kc);
  Node *node_s = reinterpret_cast<Node *>(sm + y.node);
  uint16_t *above = reinterpret_cast<uint16_t *>(sm + y.above), *pos_s = reinterpret_cast<uint16_t *>(sm + y.pos);
  int16_t *par = reinterpret_cast<int16_t *>(sm + y.par);
  uint8_t *depth = sm + y.depth;
  Entry *entries = reinterpret_cast<Entry *>(sm + y.entries);
  uint32_t *vis = reinterpret_cast<uint32_t *>(u_s);  // before a block has updates, in their place
  float *red = dots;                                  // [2][4][128]: the root's sums
  float *g_s = u_s;                                   // before there are updates

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&fx.mma, 1);
    mbar_init(&fx.drain, 1);
    fx.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&fx.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  block_sync();
  tc_fence_after();
  const uint32_t tmem = fx.tmem;
  // not before the block has its tensor memory (see delta_chunk.cu)
  pdl_launch_dependents();
  pdl_wait();

  const int l = tid & 127, d0 = (tid >> 7) * 32;  // of the state: its column, the lane of tensor memory, and 32 rows
  const uint32_t me = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  constexpr uint32_t id = idesc_16<T>(128, C, false), id2 = idesc_16<T>(128, 128, false);
  const int steps = p.Dk / 16;
  bool ok = true;
  uint32_t n_mma = 0;
  volatile int *abort_flag = &fx.abort;
  // All wait for the products that were issued.
  auto wait_products = [&]() {
    if (ok && !mbar_wait(&fx.mma, n_mma & 1u, abort_flag)) {
      ok = false;
      if (!*abort_flag) report(p.status, MFD_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    ++n_mma;
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
  };

  // A block takes a stretch of all (request, head, slice) items: mostly heads of one
  // request, whose tree is sorted once.
  const int items = p.n_req * p.Hv * slices;
  const int item0 = (int)((int64_t)items * blockIdx.x / gridDim.x), item1 = (int)((int64_t)items * (blockIdx.x + 1) / gridDim.x);
  int request_now = -1, n = 0, nn = 0;
  int64_t tok0 = 0;
  Request q = {};
  for (int item = item0; item < item1; ++item) {
    const int slice = item % slices, h = item / slices % p.Hv, r = item / slices / p.Hv;
    const int hk = h / (p.Hv / p.Hk), col = slice * LANES + l, c0 = slice * LANES + lane * LN;
    const bool have = l < LANES && col < p.Dv;
    if (r != request_now) {
      // ------------------------------------------------------- the tree
      request_now = r;
      q = request(p, r);
      tok0 = (int64_t)r * p.N;
      nn = q.ok ? q.nn : 0;
      block_sync();  // the request before is done with
      if (tid == 0) fx.bad = 0;
      block_sync();
      for (int i = tid; i < nn; i += THREADS) {
        const int up = __ldg(p.parent + tok0 + i);
        if (i == 0 ? up != -1 : (up < 0 || up >= i)) fx.bad = 1;
        par[i] = (int16_t)(i == 0 ? -1 : min(max(up, 0), i - 1));
      }
      block_sync();
      // depths, and how many nodes of a warp's 32 are as deep and before
      for (int base = 0; base < nn; base += THREADS) {
        const int i = base + tid;
        int d = 0;
        if (i < nn) {
          for (int j = i; j > 0 && d <= DEPTH; j = par[j]) ++d;
          if (d > DEPTH) {
            fx.bad = 1;
            d = DEPTH;
          }
          depth[i] = (uint8_t)d;
        }
        int rank = 0;
        for (int e = 1; e <= DEPTH; ++e) {
          const unsigned m = __ballot_sync(0xffffffffu, i < nn && d == e);
          if (d == e) rank = __popc(m & ((1u << lane) - 1u));
          if (lane == 0) fx.hist[e][base / 32 + warp] = __popc(m);
        }
        if (i < nn) pos_s[i] = (uint16_t)rank;
      }
      block_sync();
      if (fx.bad) nn = 0;
      if ((!q.ok || fx.bad) && tid == 0) report(p.status, MFD_ERR_INPUT);
      n = nn > 0 ? nn - 1 : 0;
      if (n > 0) {
        // a depth a warp: where its nodes and each 32 of them start
        const int used = (nn + 31) / 32, e = warp + 1;  // counts: 17 at most
        const int own = lane < used ? fx.hist[e][lane] : 0;
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += up;
        }
        fx.hist[e][lane] = sum - own;
        if (lane == 31) fx.count[e] = sum;
        block_sync();
        int start = lane >= 1 && lane < e ? fx.count[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) start += __shfl_xor_sync(0xffffffffu, start, o);
        if (lane == 0) {
          fx.level[e] = start;
          if (e == DEPTH) fx.level[DEPTH + 1] = start + fx.count[DEPTH];
        }
        block_sync();
        for (int i = tid; i < nn; i += THREADS)
          if (i > 0) {
            const int d = depth[i], at = fx.level[d] + fx.hist[d][i >> 5] + pos_s[i];
            node_s[at].at = i | (d << 16);
            pos_s[i] = (uint16_t)at;
          }
        block_sync();
        for (int i = tid; i < n; i += THREADS) {
          const int at = node_s[i].at;
          int j = par[at & 0xFFFF];
          for (int e = (at >> 16) - 2; e >= 0; --e, j = par[j]) above[i * DEPTH + e] = pos_s[j];
        }
      }
    }
    // rows that are not live
    if (c0 < p.Dv)
      for (int i = nn + warp; i < p.N; i += WARPS) {
        uint16_t *to = p.out + ((tok0 + i) * p.Hv + h) * p.Dv + c0;
        if (LN == 4)
          *reinterpret_cast<uint2 *>(to) = make_uint2(0, 0);
        else
          *reinterpret_cast<uint32_t *>(to) = 0u;
      }
    if (nn == 0) continue;

    // --------------------------------------------------------- the head
    float s[32];
    {
      const float *from = p.s + (((int64_t)q.src * p.Hv + h) * p.Dk + d0) * p.Dv + col;
      const bool some = q.src >= 0 && have;
#pragma unroll
      for (int d = 0; d < 32; ++d) s[d] = some && d0 + d < p.Dk ? __ldg(from + (int64_t)d * p.Dv) : 0.f;
      if (tid == 0 && q.src >= 0 && slice == slices - 1 && h + 1 < p.Hv && item + 1 < item1)  // the next one, to L2
        bulk_prefetch_l2(p.s + ((int64_t)q.src * p.Hv + h + 1) * p.Dk * p.Dv, (uint32_t)(p.Dk * p.Dv * 4));
    }
    block_sync();  // the head before is done with; the tree is there
    // 64 rows of keys or queries from sorted place `first` on, swizzled, to rows `row0` on
    // of blocks of `rows` rows
    auto load_rows = [&](const uint16_t *from, int64_t stride, int first, uint8_t *to, int row0, int rows) {
      for (int i = tid; i < C * 16; i += THREADS) {
        const int row = i >> 4, ch = i & 15;
        uint8_t *dst = to + (ch >> 3) * (rows * 128) + (row0 + row) * 128 + (((ch & 7) ^ (row & 7)) << 4);
        if (first + row < n && ch * 8 < p.Dk)
          cp_async16(smem_u32(dst), from + (tok0 + (node_s[first + row].at & 0xFFFF)) * stride + hk * p.Dk + ch * 8);
        else
          *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
      }
    };
    if (n > 0) {
      load_rows(p.k, p.k_stride, 0, tile, 0, 128);
      load_rows(p.q, p.q_stride, 0, tile, 64, 128);
    }
    for (int i = tid; i < n; i += THREADS) {
      const int64_t at = (tok0 + (node_s[i].at & 0xFFFF)) * p.Hv + h;
      const float g = __ldg(p.g + at);
      g_s[i] = g < LEAST_LOG ? LEAST_LOG : g;
      node_s[i].beta = __ldg(p.beta + at);
      node_s[i].rk = node_s[i].rq = 1.f;
    }
    // the root's key and query
    if (warp == ISSUER) {
      float a[4], b[4], kk = 0.f, qq = 0.f, kq = 0.f;
      uint2 kr = make_uint2(0, 0), qr = kr;
      if (lane * 4 < p.Dk) {
        kr = *reinterpret_cast<const uint2 *>(p.k + tok0 * p.k_stride + hk * p.Dk + lane * 4);
        qr = *reinterpret_cast<const uint2 *>(p.q + tok0 * p.q_stride + hk * p.Dk + lane * 4);
      }
      float2 x = unpack2<T>(kr.x), z = unpack2<T>(kr.y);
      a[0] = x.x, a[1] = x.y, a[2] = z.x, a[3] = z.y;
      x = unpack2<T>(qr.x), z = unpack2<T>(qr.y);
      b[0] = x.x, b[1] = x.y, b[2] = z.x, b[3] = z.y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        kk = fmaf(a[e], a[e], kk);
        qq = fmaf(b[e], b[e], qq);
      }
      const float fk = p.normalize ? rsqrtf(warp_sum(kk) + p.eps) : 1.f, fq = p.normalize ? rsqrtf(warp_sum(qq) + p.eps) : 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        fx.k0[lane * 4 + e] = a[e] * fk;
        fx.q0[lane * 4 + e] = b[e] * fq;
        kq = fmaf(a[e] * fk, b[e] * fq, kq);
      }
      kq = warp_sum(kq);
      if (lane == 0) {
        fx.root[0] = expf(__ldg(p.g + tok0 * p.Hv + h));
        fx.root[1] = __ldg(p.beta + tok0 * p.Hv + h);
        fx.root[2] = kq;
      }
    }
    const float v0 = have ? to_float<T>(p.v[tok0 * p.v_stride + h * p.Dv + col]) : 0.f;
    block_sync();
    {  // the root: sums over this thread's rows of the state
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int d = 0; d < 32; ++d) {
        a = fmaf(fx.k0[d0 + d], s[d], a);
        b = fmaf(fx.q0[d0 + d], s[d], b);
      }
      red[(tid >> 7) * 128 + l] = a;
      red[512 + (tid >> 7) * 128 + l] = b;
    }
    for (int i = tid; i < n; i += THREADS) {  // sums of log2 decays from below the root, as two floats
      const int d = node_s[i].at >> 16;
      Two c = two_product(g_s[i], LOG2E_HI, LOG2E_LO);
      for (int e = 0; e < d - 1; ++e) c = two_sum(c, two_product(g_s[above[i * DEPTH + e]], LOG2E_HI, LOG2E_LO));
      node_s[i].chi = c.hi;
      node_s[i].clo = c.lo;
    }
    block_sync();
    {
      const float ks = red[l] + red[128 + l] + (red[256 + l] + red[384 + l]);
      const float qs = red[512 + l] + red[640 + l] + (red[768 + l] + red[896 + l]);
      const float decay = fx.root[0], u = fx.root[1] * fmaf(-decay, ks, v0);
#pragma unroll
      for (int d = 0; d < 32; ++d) s[d] = fmaf(fx.k0[d0 + d], u, decay * s[d]);
      if (have && tid < 128)
        p.out[(tok0 * p.Hv + h) * p.Dv + col] = (uint16_t)pack2<T>(p.scale * fmaf(fx.root[2], u, decay * qs), 0.f);
    }
    if (n == 0) continue;
    // the state's parts
    float back = 1.f;
    {
      uint32_t part[16];
      if (BF16) {
#pragma unroll
        for (int t = 0; t < PARTS; ++t) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint32_t a = __float_as_uint(s[2 * e]), b = __float_as_uint(s[2 * e + 1]);
            part[e] = __byte_perm(a, b, 0x7632);
            s[2 * e] -= __uint_as_float(a & 0xFFFF0000u);
            s[2 * e + 1] -= __uint_as_float(b & 0xFFFF0000u);
          }
          if (ok) tmem_st16(me + TM_S + t * 64 + d0 / 2, part);
        }
      } else {
        float top = 0.f;
#pragma unroll
        for (int d = 0; d < 32; d += 2) top = max_nan(top, s[d], s[d + 1]);
        block_sync();  // the sums are read
        red[(tid >> 7) * 128 + l] = top;
        block_sync();
        top = max_nan(max_nan(red[l], red[128 + l], red[256 + l]), red[384 + l], 0.f);
        const float up = power_for(top, 11, back);
        uint32_t lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) halves(s[2 * e] * up, s[2 * e + 1] * up, part[e], lo[e]);
        if (ok) {
          tmem_st16(me + TM_S + d0 / 2, part);
          tmem_st16(me + TM_S + 64 + d0 / 2, lo);
        }
      }
      tmem_wait_st();
    }

    for (int b0 = 0; b0 < n; b0 += C) {
      // ------------------------------------------------------- a block
      const int live = min(C, n - b0);
      uint32_t *vis_b = vis + (size_t)b0 * LANES;  // in the place of the block's updates
      if (b0) {
        block_sync();  // the block before is done with
        load_rows(p.k, p.k_stride, b0, tile, 0, 128);
        load_rows(p.q, p.q_stride, b0, tile, 64, 128);
      }
      cp_async_wait();
      fence_async_smem();
      tc_fence_before();
      block_sync();
      if (warp == ISSUER) {  // the diagonal block's dot products, and those with the state
        if (elect_one() && ok) {
          tc_fence_after();
          const uint32_t a = desc_lo(smem_u32(tile), 16);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < steps) {
              const uint32_t at = (k >> 2) * (HALF >> 4) + (k & 3) * 2;
              mma_ss(tmem + TM_G, a + at, a + at, id, k != 0);
            }
          tc_commit(&fx.mma);
#pragma unroll
          for (int t = 0; t < PARTS; ++t)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < steps) mma_ts(tmem + TM_X, tmem + TM_S + t * 64 + k * 8, a + (k >> 2) * (HALF >> 4) + (k & 3) * 2, id2, t != 0 || k != 0);
        }
        __syncwarp();
      }
      // the nodes above as bits over sorted places: four threads a row, 128 places each
      if (tid < 4 * C) {
        const int row = tid >> 2, at = b0 + row, from = (tid & 3) * 128;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (row < live) {
          const int d = node_s[at].at >> 16;
          auto set = [&](int j) {
            const uint32_t bit = 1u << (j & 31);
            const int k = (j - from) >> 5;
            w[0] |= k == 0 ? bit : 0u;
            w[1] |= k == 1 ? bit : 0u;
            w[2] |= k == 2 ? bit : 0u;
            w[3] |= k == 3 ? bit : 0u;
          };
          for (int e = 0; e < d - 1; ++e) set(above[at * DEPTH + e]);
          set(at);
        }
        if (row < live)
#pragma unroll
          for (int k = 0; k < 4; ++k) vis_b[row * 16 + (tid & 3) * 4 + k] = w[k];
      }
      if (p.normalize) {  // factors, four threads a row
        const int row = tid >> 2, part = tid & 3;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ch = part * 4 + e;
          float x[8];
          unpack8<T>(*reinterpret_cast<const uint4 *>(tile + (ch >> 3) * HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4)), x);
#pragma unroll
          for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
        }
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        const int i = row & 63;
        if (part == 0 && i < live) (row < C ? node_s[b0 + i].rk : node_s[b0 + i].rq) = rsqrtf(ss + p.eps);
      }
      block_sync();  // the bits are there
      // dot products with this block's keys, then with those of the blocks before
      for (int b1 = b0; b1 >= 0; b1 -= C) {
        if (b1 < b0) {
          load_rows(p.k, p.k_stride, b1, kc, 0, C);
          cp_async_wait();
          fence_async_smem();
          tc_fence_before();
          block_sync();
          if (warp == ISSUER) {
            if (elect_one() && ok) {
              tc_fence_after();
              const uint32_t a = desc_lo(smem_u32(tile), 16), b = desc_lo(smem_u32(kc), 16);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (k < steps) mma_ss(tmem + TM_G, a + (k >> 2) * (HALF >> 4) + (k & 3) * 2, b + (k >> 2) * (C * 128 >> 4) + (k & 3) * 2, id, k != 0);
              tc_commit(&fx.mma);
            }
            __syncwarp();
          }
        }
        wait_products();
        if (ok) {
          const int row = l & 63, j0 = (tid >> 7) * 16;
          const uint32_t bits = row < live ? vis_b[row * 16 + ((b1 + j0) >> 5)] >> (j0 & 16) & 0xFFFFu : 0u;
          if (__any_sync(0xffffffffu, bits != 0)) {
            uint32_t x[16];
            tmem_ld16(me + TM_G + j0, x);
            tmem_wait_ld();
            tie16(x);
            int slot[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) slot[e] = b1 + j0 + e < n ? (node_s[b1 + j0 + e].at >> 16) - 1 : 0;
            float *to = dots + (l >= 64 ? C * DS : 0) + row * DS;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if ((bits >> e) & 1u) to[slot[e]] = __uint_as_float(x[e]);
          }
        }
        tc_fence_before();
        block_sync();  // tensor memory and the keys are read
      }
      // the values come in over the keys; every sum's entries are made
      for (int i = tid; i < C * (LANES / 8); i += THREADS) {
        const int row = i / (LANES / 8), ch = i % (LANES / 8), c = slice * LANES + ch * 8;
        if (row < live && c < p.Dv)
          cp_async16(smem_u32(v_s + row * LANES + ch * 8),
                     p.v + (tok0 + (node_s[b0 + row].at & 0xFFFF)) * p.v_stride + h * p.Dv + c);
      }
      if (warp == ISSUER) {
        if (elect_one() && ok) tc_commit(&fx.mma);
        __syncwarp();
      }
      wait_products();
#pragma unroll
      for (int i = tid; i < C * DEPTH; i += THREADS) {
        const int row = i >> 4, e = i & 15;
        if (row >= live) continue;
        const Node x = node_s[b0 + row];
        const int d = x.at >> 16;
        if (e >= d) continue;
        Entry en;
        if (e < d - 1) {
          const int j = above[(b0 + row) * DEPTH + e];
          const Node z = node_s[j];
          const float w = ex2((x.chi - z.chi) + (x.clo - z.clo)) * z.rk;
          en.a = -(x.beta * x.rk * dots[row * DS + e] * w);
          en.b = dots[C * DS + row * DS + e] * w;
          en.at = j * LANES;
        } else {
          en.a = ex2(x.chi + x.clo);
          en.b = dots[C * DS + row * DS + e] * x.rk;
          en.at = 0;
        }
        entries[i] = en;
      }
      // products with the state to shared memory
      if (ok && l < LANES) {
        const int w = tid >> 7;
        uint32_t x[32];
        tmem_ld32(me + TM_X + w * 32, x);
        tmem_wait_ld();
        tie32(x);
        float *to = w < 2 ? u_s + (b0 + w * 32) * LANES + l : xq + (w - 2) * 32 * LANES + l;
        const int rows = w < 2 ? live - w * 32 : C;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e < rows) to[e * LANES] = BF16 ? __uint_as_float(x[e]) : __uint_as_float(x[e]) * back;
      }
      tc_fence_before();
      cp_async_wait();

      // level by level
      const int first_level = node_s[b0].at >> 16, last_level = node_s[b0 + live - 1].at >> 16;
      for (int e = first_level; e <= last_level; ++e) {
        block_sync();  // what the level takes is there
        const int hi = min(fx.level[e + 1], b0 + live);
        for (int i = max(fx.level[e], b0) + warp; i < hi; i += WARPS) {
          const int row = i - b0;
          const Entry *mine = entries + row * DEPTH;
          const Node x = node_s[i];
          const Entry self = mine[e - 1];
          float u[LN], o[LN], v[LN];
          if (LN == 4) {
            const uint2 w = *reinterpret_cast<const uint2 *>(v_s + row * LANES + lane * LN);
            const float2 a = unpack2<T>(w.x), b = unpack2<T>(w.y);
            v[0] = a.x, v[1] = a.y, v[LN - 2] = b.x, v[LN - 1] = b.y;
            const float4 f = *reinterpret_cast<const float4 *>(u_s + i * LANES + lane * LN);
            u[0] = f.x, u[1] = f.y, u[LN - 2] = f.z, u[LN - 1] = f.w;
            const float4 g = *reinterpret_cast<const float4 *>(xq + row * LANES + lane * LN);
            o[0] = g.x, o[1] = g.y, o[LN - 2] = g.z, o[LN - 1] = g.w;
          } else {
            const float2 a = unpack2<T>(*reinterpret_cast<const uint32_t *>(v_s + row * LANES + lane * LN));
            v[0] = a.x, v[1] = a.y;
            const float2 f = *reinterpret_cast<const float2 *>(u_s + i * LANES + lane * LN);
            u[0] = f.x, u[1] = f.y;
            const float2 g = *reinterpret_cast<const float2 *>(xq + row * LANES + lane * LN);
            o[0] = g.x, o[1] = g.y;
          }
#pragma unroll
          for (int k = 0; k < LN; ++k) {
            u[k] = x.beta * fmaf(-self.a * x.rk, u[k], v[k]);
            o[k] *= self.a;
          }
#pragma unroll 4
          for (int t = 0; t < e - 1; ++t) {
            const Entry en = mine[t];
            float w[LN];
            if (LN == 4) {
              const float4 f = *reinterpret_cast<const float4 *>(u_s + en.at + lane * LN);
              w[0] = f.x, w[1] = f.y, w[LN - 2] = f.z, w[LN - 1] = f.w;
            } else {
              const float2 f = *reinterpret_cast<const float2 *>(u_s + en.at + lane * LN);
              w[0] = f.x, w[1] = f.y;
            }
#pragma unroll
            for (int k = 0; k < LN; ++k) {
              u[k] = fmaf(en.a, w[k], u[k]);
              o[k] = fmaf(en.b, w[k], o[k]);
            }
          }
          const float f = p.scale * x.rq;
          if (LN == 4)
            *reinterpret_cast<float4 *>(u_s + i * LANES + lane * LN) = make_float4(u[0], u[1], u[LN - 2], u[LN - 1]);
          else
            *reinterpret_cast<float2 *>(u_s + i * LANES + lane * LN) = make_float2(u[0], u[1]);
#pragma unroll
          for (int k = 0; k < LN; ++k) o[k] = f * fmaf(self.b, u[k], o[k]);
          if (c0 < p.Dv && ok) {
            uint16_t *to = p.out + ((tok0 + (x.at & 0xFFFF)) * p.Hv + h) * p.Dv + c0;
            if (LN == 4)
              *reinterpret_cast<uint2 *>(to) = make_uint2(pack2<T>(o[0], o[1]), pack2<T>(o[LN - 2], o[LN - 1]));
            else
              *reinterpret_cast<uint32_t *>(to) = pack2<T>(o[0], o[1]);
          }
        }
      }
    }
  }
  // no product runs on when tensor memory is given back
  if (warp == ISSUER) {
    if (elect_one()) {
      tc_commit(&fx.drain);
      int never = 0;
      mbar_wait(&fx.drain, 0, &never);
    }
    __syncwarp();
  }
  tc_fence_before();
  block_sync();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <typename T, int LN>
cudaError_t launch_lanes(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};  // devices this kernel is set up on
  if (dev > 63 || !((ready.load(std::memory_order_relaxed) >> dev) & 1u)) {
    if ((e = cudaFuncSetAttribute(delta_tree_kernel<T, LN>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448)) != cudaSuccess)
      return e;
    if (dev < 64) ready.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  }
  const int slices = (A.Dv + 32 * LN - 1) / (32 * LN);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int64_t items = (int64_t)A.n_req * A.Hv * slices;
  cfg.gridDim = dim3((unsigned)(items < n_sm ? items : n_sm));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)layout(A.N, 32 * LN).total + 1024;
  cfg.stream = stream;
  e = cudaLaunchKernelEx(&cfg, delta_tree_kernel<T, LN>, A, slices);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  return lanes_for(A.N) == 128 ? launch_lanes<T, 4>(A, n_sm, stream) : launch_lanes<T, 2>(A, n_sm, stream);
}

}  // namespace

cudaError_t launch_delta_tree(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  return A.dtype == MFD_BF16 ? launch_type<__nv_bfloat16>(A, n_sm, stream) : launch_type<__half>(A, n_sm, stream);
}

}  // namespace mfd
