// delta_tree.cu -- the gated delta rule over a tree's nodes, each behind its own
// path, from a state that stays (the method's pages name tree kernels for hybrid
// targets: model card "MFD drafter for Qwen3.5-4B", Usage).
//
// Unrolled along a path, a node's update is a sum over the nodes above it, at
// most 16.  The root is done first, into the state that all others start from;
// for a node i below it, with c the sum of g along its path and r, s the factors
// that the norms give its key and query,
//
//   u_i = b_i - sum_{j above i} A_ij u_j,   b_i = beta_i (v_i - e^(c_i) r_i S^T k_i)
//   A_ij = beta_i r_i r_j e^(c_i - c_j) (k_i . k_j)
//   o_i = scale s_i (e^(c_i) S^T q_i + sum_{j above i, or i} P_ij u_j)
//   P_ij = r_j e^(c_i - c_j) (q_i . k_j)
//
// Of the updates only the outputs' sums are wanted: with W = P (I + A)^-1,
//
//   o_i = scale s_i (e^(c_i) S^T q_i + sum_{j above i, or i} W_ij b_j)
//
// and row i of W is a substitution along i's path alone, half a warp's work
// without the values' columns.  So no node waits for another: there are no
// levels, and what a node holds reaches no node beside it.
//
// The products with the state, and of queries and keys with keys, are 64 nodes
// at a time on the tensor cores, issued by a warp of its own.  Nodes are sorted
// by depth, so that a node's path is in its block and the ones before.
//
// Keys and queries go to the tensor cores as they are.  The state goes in as a
// sum of numbers of their type: three of bf16, each the front of what is left
// (24 bits), or two of fp16 after a power of two for each column, which brings its
// largest to [2^14, 2^15) (22 bits of what is at least 2^-17 of that; 2^-39 of the
// largest below).
//
// 32 trees of 129 nodes and 32 heads of 128 x 128 take 134 us, a head some 36,000
// cycles of an SM: a third until its state and rows have come and the root is done,
// the rest phases of 1,000 to 1,500 cycles, each as long as its loads from shared
// memory and its exchanges take, with a barrier of 16 warps after it.  The tensor cores
// work 11% of the time.  (Fetching the next head's state during a head's outputs cost
// more in registers than it hid: 154 us.)
#include <atomic>
#include <type_traits>

#include "delta_tc.cuh"

namespace mfd {
namespace {

constexpr int C = 64;        // nodes of a block
constexpr int WORKERS = 512, WARPS = WORKERS / 32, THREADS = WORKERS + 32;
constexpr int DEPTH = DELTA_MAX_DEPTH;
constexpr int MAX_DK = 128;
constexpr int HALF = 128 * 128;  // 64 columns of a block's keys and queries

// Orders to the warp that issues products: a tree's first block, a later one, another
// block's keys (to the one or the other place of TM_G), no more.
enum { FIRST = 0, NEXT = 1, KEYS = 2, END = 4 };

// Tensor memory, columns.
constexpr int TM_S = 0;    // the state's parts, 64 each
constexpr int TM_X = 192;  // S^T [K; Q]^T
constexpr int TM_G = 320;  // [K; Q] K'^T of two blocks, two in turn

struct Node {
  float chi, clo, beta, rk, rq;
  int at;  // node, and its depth from bit 16
};
struct Fixed {
  uint64_t go, dot[2], x, drain;
  uint32_t tmem;
  int bad, abort, order;  // order: what the products' warp is to do
  float root[4];  // decay, beta, q . k
  int level[DEPTH + 2];
  int hist[DEPTH + 1][32], count[DEPTH + 1];
  float k0[MAX_DK], q0[MAX_DK];
  float2 rhs[C], out[C];  // of a block's nodes: factors of v and S^T k in b; of S^T q and the whole in o
};
// The rest of shared memory, by the number of nodes.
struct Layout {
  int blocks, kc, v, w, a, u, node, above, par, depth, pos, fixed, total;
};
constexpr int MOST_SMEM = 232448;
__host__ __device__ inline Layout layout(int N, int lanes) {
  const int n = N > 1 ? N - 1 : 1;
  Layout y;
  // Two blocks are loaded whole where they fit beside the rest: keys' 64 rows, then
  // queries', later S^T Q^T; the first one's keys again; values.  Else one block at a
  // time, and the values over the other block's keys.
  const int most = (n + C - 1) / C;
  for (y.blocks = most <= 2 ? most : 1;; --y.blocks) {
    int at = y.blocks * 2 * HALF;
    y.kc = at;
    at += C * 256;
    y.v = y.blocks == most ? at : y.kc;
    at += y.blocks == most ? y.blocks * C * lanes * 2 : 0;
    y.w = at;  // P, then W, of the block; and the root's sums
    at += C * DEPTH * 4;
    y.a = at;
    at += n * DEPTH * 4;
    y.u = at;  // b
    at += n * lanes * 4;
    y.node = at;
    at += n * (int)sizeof(Node);
    y.above = (at + 15) / 16 * 16;
    at = y.above + n * DEPTH * 2;
    y.par = at;
    at += (N * 2 + 15) / 16 * 16;
    y.pos = at;
    at += (N * 2 + 15) / 16 * 16;
    y.depth = at;
    at += (N + 15) / 16 * 16;
    y.fixed = (at + 15) / 16 * 16;
    y.total = y.fixed + (int)sizeof(Fixed) + 1024;  // and to a 1024-byte border
    if (y.total <= MOST_SMEM || y.blocks == 1) return y;
  }
}

template <typename T, int LN>  // LN: columns a lane has in the sums
__global__ void __launch_bounds__(THREADS, 1) delta_tree_kernel(const DeltaArgs p, int slices) {
  constexpr int LANES = 32 * LN;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int PARTS = BF16 ? 3 : 2;
  extern __shared__ uint8_t raw_smem[];
  uint8_t *sm = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  const Layout y = layout(p.N, LANES);
  Fixed &fx = *reinterpret_cast<Fixed *>(sm + y.fixed);
  uint8_t *kc = sm + y.kc;
  const bool whole = y.v != y.kc;  // all blocks are in shared memory at once
  float *w_s = reinterpret_cast<float *>(sm + y.w), *a_s = reinterpret_cast<float *>(sm + y.a);
  float *u_s = reinterpret_cast<float *>(sm + y.u);
  Node *node_s = reinterpret_cast<Node *>(sm + y.node);
  uint16_t *above = reinterpret_cast<uint16_t *>(sm + y.above), *pos_s = reinterpret_cast<uint16_t *>(sm + y.pos);
  int16_t *par = reinterpret_cast<int16_t *>(sm + y.par);
  uint8_t *depth = sm + y.depth;
  uint32_t *vis = reinterpret_cast<uint32_t *>(u_s);  // before a block has its b, in their place
  float *red = w_s;                                   // [2][4][128]: the root's sums
  float *g_s = u_s;                                   // before there is a b

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&fx.go, WARPS);
    mbar_init(&fx.dot[0], 1);
    mbar_init(&fx.dot[1], 1);
    mbar_init(&fx.x, 1);
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

  bool ok = true;
  volatile int *abort_flag = &fx.abort;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity, abort_flag)) {
      ok = false;
      if (!*abort_flag) report(p.status, MFD_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  };
  // A block takes a stretch of all (request, head, slice) items: mostly heads of one
  // request, whose tree is sorted once.
  const int items = p.n_req * p.Hv * slices;
  const int item0 = (int)((int64_t)items * blockIdx.x / gridDim.x), item1 = (int)((int64_t)items * (blockIdx.x + 1) / gridDim.x);

  if (warp == WARPS) {
    // ----------------------------------------------------------- products
    if (elect_one()) {
      constexpr uint32_t id = idesc_16<T>(128, C, false), id2 = idesc_16<T>(128, 128, false);
      const int steps = p.Dk / 16;
      const uint32_t tile0 = desc_lo(smem_u32(sm), 16), b = desc_lo(smem_u32(kc), 16);
      uint32_t a = tile0;
      for (uint32_t n_go = 0;; ++n_go) {
        wait(&fx.go, n_go & 1u);
        const int order = *(volatile int *)&fx.order;
        if (!ok || order == END) break;
        tc_fence_after();
        if (order >= KEYS) {  // dot products with the keys of a block further up
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < steps)
              mma_ss(tmem + TM_G + (order - KEYS) * C, a + (k >> 2) * (HALF >> 4) + (k & 3) * 2, b + (k >> 2) * (C * 128 >> 4) + (k & 3) * 2, id,
                     k != 0);
          tc_commit(&fx.dot[order - KEYS]);
          continue;
        }
        a = tile0 + (order == NEXT && whole ? 2 * HALF >> 4 : 0);
#pragma unroll
        for (int k = 0; k < 8; ++k)  // with the block's own
          if (k < steps) {
            const uint32_t at = (k >> 2) * (HALF >> 4) + (k & 3) * 2;
            mma_ss(tmem + TM_G, a + at, a + at, id, k != 0);
          }
        tc_commit(&fx.dot[0]);
        if (order == NEXT) {  // and with those of the block before
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < steps)
              mma_ss(tmem + TM_G + C, a + (k >> 2) * (HALF >> 4) + (k & 3) * 2, b + (k >> 2) * (C * 128 >> 4) + (k & 3) * 2, id, k != 0);
          tc_commit(&fx.dot[1]);
        }
#pragma unroll
        for (int t = 0; t < PARTS; ++t)  // S^T [K; Q]^T
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < steps)
              mma_ts(tmem + TM_X, tmem + TM_S + t * 64 + k * 8, a + (k >> 2) * (HALF >> 4) + (k & 3) * 2, id2, t != 0 || k != 0);
        tc_commit(&fx.x);
      }
      // no product runs on when tensor memory is given back
      tc_commit(&fx.drain);
      int never = 0;
      mbar_wait(&fx.drain, 0, &never);
    }
    __syncwarp();
    tc_fence_before();
    block_sync();
    tc_fence_after();
    return;
  }

  // ------------------------------------------------------------- workers
  const int l = tid & 127, d0 = (tid >> 7) * 32;  // of the state: its column, the lane of tensor memory, and 32 rows
  const uint32_t me = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  uint32_t dot_par = 0, x_par = 0;  // phases to wait for
  auto sync = [&]() { named_sync(1, WORKERS); };
  auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
    wait(bar, parity);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
  };
  // What this thread wrote is there for the products.  An order is read before the
  // next one is given: all wait for what came of it in between.
  auto go = [&](int order) {
    if (tid == 0) *(volatile int *)&fx.order = order;
    fence_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&fx.go);
  };
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
      sync();  // the request before is done with
      if (tid == 0) fx.bad = 0;
      sync();
      for (int i = tid; i < nn; i += WORKERS) {
        const int up = __ldg(p.parent + tok0 + i);
        if (i == 0 ? up != -1 : (up < 0 || up >= i)) fx.bad = 1;
        par[i] = (int16_t)(i == 0 ? -1 : min(max(up, 0), i - 1));
      }
      sync();
      // depths, and how many nodes of a warp's 32 are as deep and before
      for (int base = 0; base < nn; base += WORKERS) {
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
      sync();
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
        sync();
        int start = lane >= 1 && lane < e ? fx.count[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) start += __shfl_xor_sync(0xffffffffu, start, o);
        if (lane == 0) {
          fx.level[e] = start;
          if (e == DEPTH) fx.level[DEPTH + 1] = start + fx.count[DEPTH];
        }
        sync();
        for (int i = tid; i < nn; i += WORKERS)
          if (i > 0) {
            const int d = depth[i], at = fx.level[d] + fx.hist[d][i >> 5] + pos_s[i];
            node_s[at].at = i | (d << 16);
            pos_s[i] = (uint16_t)at;
          }
        sync();
        for (int i = tid; i < n; i += WORKERS) {
          const int at = node_s[i].at;
          int j = par[at & 0xFFFF];
          for (int e = (at >> 16) - 2; e >= 0; --e, j = par[j]) above[i * DEPTH + e] = pos_s[j];
        }
      }
    }
    sync();  // the head before is done with, the tree is there
    // rows that are not live
    if (c0 < p.Dv)
      for (int i = nn + warp; i < p.N; i += WARPS) {
        uint16_t *to = p.out + ((tok0 + i) * p.Hv + h) * p.Dv + c0;
        if (LN == 4)
          *reinterpret_cast<uint2 *>(to) = make_uint2(0, 0);
        else if (LN == 2)
          *reinterpret_cast<uint32_t *>(to) = 0u;
        else
          *to = 0;
      }
    if (nn == 0) continue;

    // --------------------------------------------------------- the head
    float own_g = 0.f, own_beta = 0.f;  // of the node that this thread looks after
    if (tid < n) {
      const int64_t at = (tok0 + (node_s[tid].at & 0xFFFF)) * p.Hv + h;
      own_g = __ldg(p.g + at);
      own_beta = __ldg(p.beta + at);
    }
    float s[32];
    {
      const float *from = p.s + (((int64_t)q.src * p.Hv + h) * p.Dk + d0) * p.Dv + col;
      const bool some = q.src >= 0 && have;
#pragma unroll
      for (int d = 0; d < 32; ++d) s[d] = some && d0 + d < p.Dk ? __ldg(from + (int64_t)d * p.Dv) : 0.f;
      if (tid == 0 && q.src >= 0 && slice == slices - 1 && h + 1 < p.Hv && item + 1 < item1)  // the next one, to L2
        bulk_prefetch_l2(p.s + ((int64_t)q.src * p.Hv + h + 1) * p.Dk * p.Dv, (uint32_t)(p.Dk * p.Dv * 4));
    }
    // A thread loads chunk `ch` of rows row16, row16 + 32 of a block: of its keys and
    // queries to `to`, of the values to `tv`, of the keys alone to `tk` (each may be NULL).
    const int ch = tid & 15, row16 = tid >> 4;
    auto load = [&](int first, uint8_t *to, uint16_t *tv, uint8_t *tk) {
      const uint32_t swizzle = ((ch & 7) ^ (row16 & 7)) << 4;
      const bool dk = ch * 8 < p.Dk, dv = ch * 8 < LANES && slice * LANES + ch * 8 < p.Dv;
#pragma unroll
      for (int row = row16; row < C; row += 32) {
        const bool there = first + row < n;
        const int64_t tok = tok0 + (there ? node_s[first + row].at & 0xFFFF : 0);
        const uint16_t *kr = p.k + tok * p.k_stride + hk * p.Dk + ch * 8;
        uint8_t *kq = to + (ch >> 3) * HALF + row * 128 + swizzle, *k1 = tk + (ch >> 3) * (C * 128) + row * 128 + swizzle;
        if (there && dk) {
          if (to) cp_async16(smem_u32(kq), kr);
          if (to) cp_async16(smem_u32(kq + C * 128), p.q + tok * p.q_stride + hk * p.Dk + ch * 8);
          if (tk) cp_async16(smem_u32(k1), kr);
        } else {
          if (to) *reinterpret_cast<uint4 *>(kq) = *reinterpret_cast<uint4 *>(kq + C * 128) = make_uint4(0, 0, 0, 0);
          if (tk) *reinterpret_cast<uint4 *>(k1) = make_uint4(0, 0, 0, 0);
        }
        if (tv && there && dv)
          cp_async16(smem_u32(tv + row * LANES + ch * 8), p.v + tok * p.v_stride + h * p.Dv + slice * LANES + ch * 8);
      }
    };
    uint16_t *const v0_s = reinterpret_cast<uint16_t *>(sm + y.v);
    for (int b0 = 0; b0 < (whole ? n : n > 0 ? 1 : 0); b0 += C)
      load(b0, sm + b0 / C * (2 * HALF), whole ? v0_s + b0 * LANES : nullptr, whole && b0 == 0 ? kc : nullptr);
    if (tid < n) {
      g_s[tid] = own_g < LEAST_LOG ? LEAST_LOG : own_g;
      node_s[tid].beta = own_beta;
      node_s[tid].rk = node_s[tid].rq = 1.f;
    }
    // the root's key and query
    if (warp == WARPS - 1) {
      float a[4], b[4], kk = 0.f, qq = 0.f, kq = 0.f;
      uint2 kr = make_uint2(0, 0), qr = kr;
      const float g0 = __ldg(p.g + tok0 * p.Hv + h), beta0 = __ldg(p.beta + tok0 * p.Hv + h);
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
        fx.root[0] = expf(g0);
        fx.root[1] = beta0;
        fx.root[2] = kq;
      }
    }
    const float v0 = have ? to_float<T>(p.v[tok0 * p.v_stride + h * p.Dv + col]) : 0.f;
    sync();
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
    for (int i = tid; i < n; i += WORKERS) {  // sums of log2 decays from below the root, as two floats
      const int d = node_s[i].at >> 16;
      const uint4 j0 = *reinterpret_cast<const uint4 *>(above + i * DEPTH), j1 = *reinterpret_cast<const uint4 *>(above + i * DEPTH + 8);
      const uint32_t js[8] = {j0.x, j0.y, j0.z, j0.w, j1.x, j1.y, j1.z, j1.w};
      // the sum of the high parts, and what each addition to it and each product lost
      Two c = two_product(g_s[i], LOG2E_HI, LOG2E_LO);
#pragma unroll
      for (int e = 0; e < DEPTH - 1; ++e) {
        const Two x = two_product(e < d - 1 ? g_s[(js[e >> 1] >> (16 * (e & 1))) & 0xFFFFu] : 0.f, LOG2E_HI, LOG2E_LO);
        const Two t = two_sum(c.hi, x.hi);
        c.hi = t.hi;
        c.lo += t.lo + x.lo;
      }
      c = two_sum(c.hi, c.lo);
      node_s[i].chi = c.hi;
      node_s[i].clo = c.lo;
    }
    sync();
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
        sync();  // the sums are read
        red[(tid >> 7) * 128 + l] = top;
        sync();
        top = max_nan(max_nan(red[l], red[128 + l], red[256 + l]), red[384 + l], 0.f);
        const float up = power_for(top, 14, back);
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
      uint32_t *vis_b = vis + (size_t)b0 * LANES;
      uint8_t *tile = sm + (whole ? b0 / C * (2 * HALF) : 0);
      float *xq = reinterpret_cast<float *>(tile);
      uint16_t *v_s = v0_s + (whole ? b0 * LANES : 0);
      if (b0 && whole) sync();
      if (b0 && !whole) {
        sync();  // the block before is done with
        load(b0, tile, nullptr, nullptr);
        load(b0 - C, nullptr, nullptr, kc);
      }
      // meanwhile the nodes above as bits over sorted places: four threads a row, 128
      // places each
      if (tid < 4 * C) {
        const int row = tid >> 2, at = b0 + row, from = (tid & 3) * 128;
        if (row < live) {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
          const int d = node_s[at].at >> 16;
          auto set = [&](int j) {
            const uint32_t bit = 1u << (j & 31);
            const int k = (j - from) >> 5;
            w[0] |= k == 0 ? bit : 0u;
            w[1] |= k == 1 ? bit : 0u;
            w[2] |= k == 2 ? bit : 0u;
            w[3] |= k == 3 ? bit : 0u;
          };
          const uint4 j0 = *reinterpret_cast<const uint4 *>(above + at * DEPTH), j1 = *reinterpret_cast<const uint4 *>(above + at * DEPTH + 8);
          const uint32_t js[8] = {j0.x, j0.y, j0.z, j0.w, j1.x, j1.y, j1.z, j1.w};
#pragma unroll
          for (int e = 0; e < DEPTH - 1; ++e)
            if (e < d - 1) set((js[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
          set(at);
          *reinterpret_cast<uint4 *>(vis_b + row * 16 + (tid & 3) * 4) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      cp_async_wait();
      go(b0 ? NEXT : FIRST);
      sync();
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
      // dot products with this block's keys, then with those of the blocks before: those
      // of keys to A, those of queries to P
      for (int b1 = b0; b1 >= 0; b1 -= C) {
        if (b0 - b1 >= 2 * C) {
          sync();  // the keys before have been used, the dot products before last read
          load(b1, nullptr, nullptr, kc);
          cp_async_wait();
          go(KEYS + ((b0 - b1) & C ? 1 : 0));
        }
        const int g = (b0 - b1) & C ? 1 : 0;
        wait_warp(&fx.dot[g], (dot_par >> g) & 1u);
        dot_par ^= 1u << g;
        if (!ok) continue;
        const int row = l & 63, j0 = (tid >> 7) * 16;
        const uint32_t bits = row < live ? vis_b[row * 16 + ((b1 + j0) >> 5)] >> (j0 & 16) & 0xFFFFu : 0u;
        if (__any_sync(0xffffffffu, bits != 0)) {
          uint32_t x[16];
          tmem_ld16(me + TM_G + g * C + j0, x);
          tmem_wait_ld();
          tie16(x);
          int slot[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) slot[e] = b1 + j0 + e < n ? (node_s[b1 + j0 + e].at >> 16) - 1 : 0;
          float *to = l >= 64 ? w_s + row * DEPTH : a_s + (b0 + row) * DEPTH;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if ((bits >> e) & 1u) to[slot[e]] = __uint_as_float(x[e]);
        }
        tc_fence_before();
      }
      sync();
      if (!whole) load(b0, nullptr, v_s, nullptr);  // over the keys
      // factors
#pragma unroll
      for (int i = tid; i < C * DEPTH; i += WORKERS) {
        const int row = i >> 4, e = i & 15;
        if (row >= live) continue;
        const Node x = node_s[b0 + row];
        const int d = x.at >> 16;
        if (e == 0) {
          const float ec = ex2(x.chi + x.clo);
          fx.rhs[row] = make_float2(x.beta, -x.beta * x.rk * ec);
          fx.out[row] = make_float2(ec, p.scale * x.rq);
        }
        if (e < d - 1) {
          const Node z = node_s[above[(b0 + row) * DEPTH + e]];
          const float w = ex2((x.chi - z.chi) + (x.clo - z.clo)) * z.rk;
          a_s[(b0 + row) * DEPTH + e] *= x.beta * x.rk * w;
          w_s[i] *= w;
        } else if (e == d - 1) {
          w_s[i] *= x.rk;
        }
      }
      cp_async_wait();
      sync();
      // W: half a warp a node, a node above it a lane; the last known element's part is
      // taken off those of the nodes above
#pragma unroll
      for (int pass = 0; pass < C / 32; ++pass) {
        const int row = pass * 32 + (tid >> 4), e = tid & 15;
        const int d = row < live ? node_s[b0 + row].at >> 16 : 0;
        const int own = e < d - 1 ? above[(b0 + row) * DEPTH + e] : b0 + row;
        float w = e < d ? w_s[row * DEPTH + e] : 0.f;
        const int most = max(d, __shfl_xor_sync(0xffffffffu, d, 16));
#pragma unroll 4
        for (int m = most - 1; m > 0; --m) {
          const int at = __shfl_sync(0xffffffffu, own, m, 16);
          const float a = m < d && e < m ? a_s[at * DEPTH + e] : 0.f;
          const float last = __shfl_sync(0xffffffffu, w, m, 16);
          if (m < d && e < m) w = fmaf(-last, a, w);
        }
        if (e < d) w_s[row * DEPTH + e] = w;
      }
      // b and S^T q to shared memory
      wait_warp(&fx.x, x_par);
      x_par ^= 1u;
      if (ok && l < LANES) {
        const int w = tid >> 7, first = (w & 1) * 32, rows = live - first;
        uint32_t x[32];
        tmem_ld32(me + TM_X + w * 32, x);
        tmem_wait_ld();
        tie32(x);
        if (!BF16)
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * back);
        if (w < 2) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float2 f = fx.rhs[first + e];
            x[e] = __float_as_uint(fmaf(f.y, __uint_as_float(x[e]), f.x * to_float<T>(v_s[(first + e) * LANES + l])));
          }
        }
        float *to = (w < 2 ? u_s + (b0 + first) * LANES : xq + first * LANES) + l;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e < rows) to[e * LANES] = __uint_as_float(x[e]);
      }
      tc_fence_before();
      sync();
      // outputs, a node half a warp: a lane has columns from c and from c + 16 LN on
      for (int row = row16; row < live; row += 32) {
        const int i = b0 + row, at = node_s[i].at, d = at >> 16, c = ch * LN;
        const float2 f = fx.out[row];
        const float *mine = w_s + row * DEPTH;
        const uint16_t *up = above + i * DEPTH;
        float o[2 * LN];
        auto take = [&](const float *from, float (&x)[2 * LN]) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float *at = from + c + e * 16 * LN;
            if (LN == 4) {
              const float4 y = *reinterpret_cast<const float4 *>(at);
              x[e * LN] = y.x, x[e * LN + (LN > 1 ? 1 : 0)] = y.y, x[e * LN + (LN > 2 ? 2 : 0)] = y.z, x[e * LN + LN - 1] = y.w;
            } else if (LN == 2) {
              const float2 y = *reinterpret_cast<const float2 *>(at);
              x[e * LN] = y.x, x[e * LN + LN - 1] = y.y;
            } else {
              x[e * LN] = *at;
            }
          }
        };
        take(xq + row * LANES, o);
        {
          float b[2 * LN];
          take(u_s + i * LANES, b);
          const float self = mine[d - 1];
#pragma unroll
          for (int k = 0; k < 2 * LN; ++k) o[k] = fmaf(self, b[k], f.x * o[k]);
        }
        int t = 0;
        for (; t + 2 <= d - 1; t += 2) {
          const float2 w = *reinterpret_cast<const float2 *>(mine + t);
          const uint32_t j = *reinterpret_cast<const uint32_t *>(up + t);
          float x[2 * LN], z[2 * LN];
          take(u_s + (j & 0xFFFFu) * LANES, x);
          take(u_s + (j >> 16) * LANES, z);
#pragma unroll
          for (int k = 0; k < 2 * LN; ++k) o[k] = fmaf(w.y, z[k], fmaf(w.x, x[k], o[k]));
        }
        if (t < d - 1) {
          float x[2 * LN];
          take(u_s + up[t] * LANES, x);
          const float w = mine[t];
#pragma unroll
          for (int k = 0; k < 2 * LN; ++k) o[k] = fmaf(w, x[k], o[k]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int cc = slice * LANES + c + e * 16 * LN;
          const float *y = o + e * LN;
          uint16_t *to = p.out + ((tok0 + (at & 0xFFFF)) * p.Hv + h) * p.Dv + cc;
          if (cc >= p.Dv || !ok) continue;
          if (LN == 4)
            *reinterpret_cast<uint2 *>(to) =
                make_uint2(pack2<T>(f.y * y[0], f.y * y[LN > 1 ? 1 : 0]), pack2<T>(f.y * y[LN > 2 ? 2 : 0], f.y * y[LN - 1]));
          else if (LN == 2)
            *reinterpret_cast<uint32_t *>(to) = pack2<T>(f.y * y[0], f.y * y[LN - 1]);
          else
            *to = (uint16_t)pack2<T>(f.y * y[0], 0.f);
        }
      }
    }
  }
  go(END);
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
    if ((e = cudaFuncSetAttribute(delta_tree_kernel<T, LN>, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST_SMEM)) != cudaSuccess)
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
  cfg.dynamicSmemBytes = (size_t)layout(A.N, 32 * LN).total;
  cfg.stream = stream;
  e = cudaLaunchKernelEx(&cfg, delta_tree_kernel<T, LN>, A, slices);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  // As many columns as fit beside all nodes, fewer where heads alone leave SMs without
  // work: a tree of 257 nodes and 32 heads takes 39 us in slices of 32 columns, 42 in
  // slices of 128; four trees of 129 take 64 and 21.
  const int64_t heads = (int64_t)A.n_req * A.Hv;
  const auto slices = [&](int lanes) { return heads * ((A.Dv + lanes - 1) / lanes); };
  if (layout(A.N, 128).total <= MOST_SMEM && slices(64) > n_sm) return launch_lanes<T, 4>(A, n_sm, stream);
  if (layout(A.N, 64).total <= MOST_SMEM && slices(32) > n_sm) return launch_lanes<T, 2>(A, n_sm, stream);
  return launch_lanes<T, 1>(A, n_sm, stream);
}

}  // namespace

cudaError_t launch_delta_tree(const DeltaArgs &A, int n_sm, cudaStream_t stream) {
  return A.dtype == MFD_BF16 ? launch_type<__nv_bfloat16>(A, n_sm, stream) : launch_type<__half>(A, n_sm, stream);
}

}  // namespace mfd
