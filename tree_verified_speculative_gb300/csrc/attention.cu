// attention.cu -- attention of a request's rows (the tree's nodes under the
// tree mask, one token, or a stretch of a prompt) over the paged cache
// (project page "Multi-Future Drafting", How it works, step 3, Figure 2 (c):
// one target pass scores every node of the tree).
//
// For one request and key head, the N nodes' G = Hq / Hk query heads are M =
// N * G rows of one product with the head's keys, so a key or value tile
// serves all of them:
//
//   S[128 x BN] = Q[128 x D] . K[BN x D]^T            (tcgen05, fp32 in TMEM)
//   m' = max(m, max S c), P = exp2(S c - m'), l += sum P      (registers)
//   O[128 x D] += P[128 x BN] . V[BN x D]    (tcgen05, P from TMEM, fp32 in TMEM)
//   out = O / l,  lse = ln 2 * (m + log2 l),  c = scale * log2 e
//
// One pass over the keys and values; scores and weights never leave the SM.
// The running maximum m is moved, and O and l scaled down, only when a row's
// maximum has grown by more than 2^8: any m gives the same quotient, and
// weights up to 2^8 lose nothing in bf16, fp16 or fp32.
//
// Streams.  Two accumulators S and O per CTA, each with a softmax warpgroup of
// its own, so that one stream's products run while the other's weights are
// computed.  Rows for two tiles of 128 ("shared"): a stream is a row tile and
// both read every key and value tile.  Rows for one tile ("alternating"): the
// streams take the key and value tiles in turn with a maximum, sum and O each,
// joined at the end.  Heads wider than 128 leave tensor memory for one O:
// one stream, with two S accumulators used in turn.
//
// Work split.  All (request, key head, row tile pair) items and their key
// tiles form one line, ordered so that the row tiles of a head, which read
// the same keys, are neighbours; every CTA takes an equal stretch of it.  An
// item cut by a border leaves its parts (O, m, l) in scratch, and join_kernel
// combines them in a fixed order.  The line is laid out from the lengths on
// the device: a short and a long request keep all SMs busy alike, and a graph
// replays with other lengths.
//
// Warps: 0 loads (TMA, one box per page and 64 columns), 1 issues the MMAs,
// 4-7 and 8-11 softmax, the last four help: they turn E4M3 tiles into the
// operand type, and, in tiles that reach past the context, clear value rows
// past the end and values that are not finite, which a product would spread
// to rows that do not see them (0 * NaN); a cleared value's node is noted and
// added back for the rows that do see it.
#include "kvcache.h"
#include "mfd_device.cuh"

namespace mfd {
namespace {

constexpr int BM = 128;
constexpr int MAX_N = 4096;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float MAX_GROWTH = 8.f;  // log2 of how far a weight may pass 1

struct Params {
  CacheView cv;
  const uint16_t *q;
  int64_t q_stride;
  int n_req, N, Hq, G, M, W32;
  int n_pair;  // row tile groups of an item line
  const int32_t *ctx_len, *n_nodes;
  const uint32_t *mask;
  float c;  // scale * log2 e
  uint16_t *out;
  float *lse;
  int32_t *status;
  float4 *part_o;   // [slot][D / 4][part_rows]
  float2 *part_ml;  // [slot][part_rows]
  int part_rows;
};

template <int DP_, bool E4M3_>
struct Shape {
  static constexpr int DP = DP_;                       // head width, padded to 64, 128 or 256
  static constexpr int NS = DP == 256 ? 1 : 2;         // streams
  static constexpr int BN = DP == 256 ? 64 : 128;      // key positions of a tile
  static constexpr int NB = DP / 64;                   // 64-column blocks of 128-byte rows
  static constexpr int Q_TILE = BM * DP * 2;
  static constexpr int STAGE = BN * DP * 2;
  static constexpr int RAW = BN * DP;                  // an E4M3 tile as it is in the cache
  static constexpr int ST = E4M3_ ? (DP == 64 ? 4 : 3) : (DP == 64 ? 8 : 5);
  static constexpr int RST = E4M3_ ? (DP == 64 ? 6 : 4) : 0;
  static constexpr int THREADS = 128 * (2 + NS);
  static constexpr int HELP_WARP = 4 + 4 * NS;
  static constexpr int TM_S = 0;                       // S accumulators; P over them
  static constexpr int TM_O = 256;
  static constexpr int CODES = E4M3_ ? 2 * 8 * 128 : 0;
  static constexpr int BARS = 2 * ST + ST + 2 * (RST ? RST : 1) + 2 + 2 + 2 + 1 + 1;
  static constexpr int SMEM = NS * Q_TILE + ST * STAGE + RST * RAW + CODES + MAX_N / 8 + BARS * 8 + 64;
};

// ------------------------------------------------------------------ line of work

// Lengths of request q; a request whose lengths leave the cache has none.
__device__ __forceinline__ bool lengths(const Params &p, int q, int &ctx, int &nn) {
  ctx = __ldg(p.ctx_len + q);
  nn = p.n_nodes ? __ldg(p.n_nodes + q) : p.N;
  const bool ok = ctx >= 0 && nn >= 0 && nn <= p.N &&
                  (int64_t)ctx + nn <= ((int64_t)p.cv.max_pages << p.cv.ps_shift);
  if (!ok) ctx = nn = 0;
  return ok;
}

struct Item {
  int active;  // row tiles with live rows
  int tiles;   // key tiles
  int cost;    // places on the line: a step per row tile and key tile, and one for its start and end
};

template <int NS, int BN>
__device__ __forceinline__ Item item_of(const Params &p, int ctx, int nn, int pair) {
  Item it;
  const int live = nn * p.G, first = pair * NS * BM;
  it.active = live > first ? (NS == 2 && live > first + BM ? 2 : 1) : 0;
  int len = ctx + nn;
  if (!p.mask && it.active) {  // causal: nothing past the group's last row
    const int last = (live < first + NS * BM ? live : first + NS * BM) - 1;
    len = ctx + last / p.G + 1;
  }
  it.tiles = it.active ? (len + BN - 1) / BN : 0;
  it.cost = it.active * it.tiles + 1;
  return it;
}

template <int NS, int BN>
__device__ __forceinline__ int64_t head_cost(const Params &p, int ctx, int nn) {
  if (p.mask) {
    const int live = nn * p.G;
    return (int64_t)((live + BM - 1) / BM) * (nn ? (ctx + nn + BN - 1) / BN : 0) + p.n_pair;
  }
  int64_t c = 0;
  for (int i = 0; i < p.n_pair; ++i) c += item_of<NS, BN>(p, ctx, nn, i).cost;
  return c;
}

// First key tile at or after place z of an item.
__device__ __forceinline__ int tile_at(const Item &it, int z) {
  return z >= it.cost ? it.tiles : (int)((int64_t)z * it.tiles / it.cost);
}

// A CTA's stretch of one item.
struct Segment {
  int q, h, pair;
  int ctx, nn;
  Item it;
  int t0, t1;  // key tiles
  bool head;   // starts at the item's start
};

// Walks a CTA's stretch [x, x1) of the line.  Every role walks it by itself.
template <int NS, int BN>
struct Walk {
  int64_t x, x1;
  int q, h, pair, z;
  int ctx, nn;

  __device__ __forceinline__ void start(const Params &p, int64_t x_, int64_t x1_, int q0, int64_t into) {
    x = x_;
    x1 = x1_;
    q = q0;
    h = pair = z = 0;
    if (x >= x1) return;
    lengths(p, q, ctx, nn);
    const int64_t hc = head_cost<NS, BN>(p, ctx, nn);
    h = (int)(into / hc);
    int64_t rest = into - h * hc;
    for (;;) {
      const int c = item_of<NS, BN>(p, ctx, nn, pair).cost;
      if (rest < c) break;
      rest -= c;
      ++pair;
    }
    z = (int)rest;
  }
  __device__ __forceinline__ bool next(const Params &p, Segment &s) {
    if (x >= x1) return false;
    s.q = q;
    s.h = h;
    s.pair = pair;
    s.ctx = ctx;
    s.nn = nn;
    s.it = item_of<NS, BN>(p, ctx, nn, pair);
    const int64_t left = x1 - x;
    const int end = left < s.it.cost - z ? z + (int)left : s.it.cost;
    s.t0 = tile_at(s.it, z);
    s.t1 = tile_at(s.it, end);
    s.head = z == 0;
    x += end - z;
    z = 0;
    if (end == s.it.cost && ++pair == p.n_pair) {
      pair = 0;
      if (++h == p.cv.Hk) {
        h = 0;
        if (++q < p.n_req) lengths(p, q, ctx, nn);
      }
    }
    return true;
  }
};

// Where the line's place x falls: CTA c of n has [C c / n, C (c + 1) / n).
__device__ __forceinline__ int64_t border(int64_t total, int c, int n) { return total * c / n; }
__device__ __forceinline__ int cta_of(int64_t total, int64_t x, int n) { return (int)(((x + 1) * n - 1) / total); }

// ------------------------------------------------------------------ primitives

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
template <int R>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands, fp32 accumulate.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 columns of the warp's 32 lanes; valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Ties registers loaded before a wait to the code after it.
__device__ __forceinline__ void tie32(uint32_t *r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31]));
}
// The same for 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tie16(uint32_t *r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Operand descriptor of a [tokens][64 columns] block array as an operand whose
// contiguous dimension is not the contraction (the values: contraction over
// tokens).  128-byte swizzle; 64-column blocks `block_bytes` apart (leading
// byte offset), 8-token groups 1024 bytes apart (stride byte offset).
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t block_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(block_bytes >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// Instruction descriptor, kind::f16, fp32 accumulator: operand type code at
// bits 7 and 10 (0 fp16, 1 bf16), bit 16 set when B's contraction is not its
// contiguous dimension, N >> 3 at bit 17, M >> 4 at bit 24.
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc_16(int M, int N, bool b_mn);
template <>
__device__ __forceinline__ constexpr uint32_t idesc_16<__nv_bfloat16>(int M, int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
template <>
__device__ __forceinline__ constexpr uint32_t idesc_16<__half>(int M, int N, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bits of two 16-bit elements whose exponent is all ones (NaN, infinity).
template <typename T>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w);
template <>
__device__ __forceinline__ uint32_t nonfinite2<__nv_bfloat16>(uint32_t w) {
  return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u;
}
template <>
__device__ __forceinline__ uint32_t nonfinite2<__half>(uint32_t w) {
  return ((w & 0x7FFF7FFFu) + 0x04000400u) & 0x80008000u;
}

// Four E4M3 bytes to four 16-bit values times 2^e (code = e + 127, not NaN).
template <typename T>
struct Widen;
// bf16: the byte's exponent and mantissa bits moved to bf16's places read as
// the value times 2^-120 (biases 7 and 127), subnormals included; one exact
// multiplication puts both powers right, or two where 2^(e + 120) has no bf16.
template <>
struct Widen<__nv_bfloat16> {
  __nv_bfloat162 f1, f2;
  bool two;
  __device__ __forceinline__ explicit Widen(int code) {
    two = code > 134;
    const uint32_t a = two ? 247u << 7 : (uint32_t)(code + 120) << 7, b = (uint32_t)code << 7;
    const uint32_t aa = a | (a << 16), bb = b | (b << 16);
    f1 = *reinterpret_cast<const __nv_bfloat162 *>(&aa);
    f2 = *reinterpret_cast<const __nv_bfloat162 *>(&bb);
  }
  __device__ __forceinline__ uint2 operator()(uint32_t x) const {
    uint2 o;
    uint32_t y = __byte_perm(x, 0, 0x1404);
    y = (y & 0x80008000u) | ((y & 0x7F007F00u) >> 4);
    __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&y), f1);
    uint32_t w = __byte_perm(x, 0, 0x3424);
    w = (w & 0x80008000u) | ((w & 0x7F007F00u) >> 4);
    __nv_bfloat162 u = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w), f1);
    if (two) {
      v = __hmul2(v, f2);
      u = __hmul2(u, f2);
    }
    o.x = *reinterpret_cast<const uint32_t *>(&v);
    o.y = *reinterpret_cast<const uint32_t *>(&u);
    return o;
  }
};
// fp16: E4M3 converts exactly; the power is applied in fp32.
template <>
struct Widen<__half> {
  float s;
  __device__ __forceinline__ explicit Widen(int code) { s = e4m3_scale(code); }
  __device__ __forceinline__ uint2 operator()(uint32_t x) const {
    const float2 a = e4m3x2_float(x & 0xFFFFu), b = e4m3x2_float(x >> 16);
    return make_uint2(pack2<__half>(a.x * s, a.y * s), pack2<__half>(b.x * s, b.y * s));
  }
};

// Visible key positions t, t + 1, .., t + 31 of row `node`, as bits; b = t - ctx.
__device__ __forceinline__ uint32_t visible32(const uint32_t *row, int W32, int node, int nn, int b) {
  if (b + 32 <= 0) return 0xFFFFFFFFu;
  if (!row) {  // causal
    const int n = node - b + 1;
    return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
  }
  const int left = nn - b;
  if (left <= 0) return 0u;
  const int i = b >> 5;
  const uint32_t lo = i < 0 ? 0xFFFFFFFFu : __ldg(row + i);
  const uint32_t hi = i + 1 < W32 ? __ldg(row + i + 1) : 0u;
  const uint32_t w = __funnelshift_r(lo, hi, b & 31);
  return left >= 32 ? w : w & ((1u << left) - 1u);
}

// ------------------------------------------------------------------ kernel

template <typename T, int DP, bool E4M3>
__global__ void __launch_bounds__((Shape<DP, E4M3>::THREADS), 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const Params p) {
  using SH = Shape<DP, E4M3>;
  constexpr int NS = SH::NS, BN = SH::BN, NB = SH::NB, ST = SH::ST, RST = SH::RST;
  constexpr uint32_t RN = RST ? RST : 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem;
  uint8_t *sT = sQ + NS * SH::Q_TILE;
  uint8_t *sR = sT + ST * SH::STAGE;
  uint8_t *sC = sR + RST * SH::RAW;  // exponent bytes [k, v][8 tiles][128]
  uint32_t *bad = reinterpret_cast<uint32_t *>(sC + SH::CODES);
  uint64_t *full = reinterpret_cast<uint64_t *>(bad + MAX_N / 32);
  uint64_t *empty = full + ST;
  uint64_t *special = empty + ST;  // a tile the helpers go over before it is full
  uint64_t *raw_full = special + ST;
  uint64_t *raw_empty = raw_full + (RST ? RST : 1);
  uint64_t *s_full = raw_empty + (RST ? RST : 1);
  uint64_t *p_full = s_full + 2;
  uint64_t *pv_done = p_full + 2;
  uint64_t *q_full = pv_done + 2;
  uint64_t *drain = q_full + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *never = abort_flag + 1;
  volatile int *seg_done = never + 1;  // segments a softmax warpgroup has left [NS]
  int *start_q = const_cast<int *>(seg_done) + 2;
  volatile int *any_bad = start_q + 1;
  int64_t *start_x = reinterpret_cast<int64_t *>(start_q + 2 + 1);  // [x, x1, into the request]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const CacheView &cv = p.cv;

  if (smem_u32(smem) & 1023u) {  // the swizzled tiles start on 1024-byte borders
    if (tid == 0) report(p.status, MFD_ERR_CUDA);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], E4M3 ? 4 : 1);
      mbar_init(&empty[i], 1);
      mbar_init(&special[i], 1);
    }
    for (int i = 0; i < RST; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, 4 * NS);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never = 0;
    seg_done[0] = seg_done[1] = 0;
    *any_bad = 0;
    fence_mbar_init();
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // Where this CTA's stretch starts: the requests' costs, summed by warp 0
  // (in the space of the first tile, before any load is issued).
  int64_t *cost_s = reinterpret_cast<int64_t *>(sT);
  for (int q = tid; q < p.n_req; q += SH::THREADS) {
    int ctx, nn;
    if (!lengths(p, q, ctx, nn) && blockIdx.x == 0) report(p.status, MFD_ERR_INPUT);
    cost_s[q] = cv.Hk * head_cost<NS, BN>(p, ctx, nn);
  }
  block_sync();
  if (warp == 0) {
    int64_t total = 0;
    for (int q = lane; q < p.n_req; q += 32) total += cost_s[q];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int64_t x = border(total, blockIdx.x, gridDim.x), x1 = border(total, blockIdx.x + 1, gridDim.x);
    if (lane == 0) {
      start_x[0] = x;
      start_x[1] = x1;
    }
    int64_t before = 0;
    for (int q0 = 0; q0 < p.n_req; q0 += 32) {
      const int64_t own = q0 + lane < p.n_req ? cost_s[q0 + lane] : 0;
      int64_t run = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
      }
      const int64_t lo = before + run - own;
      if (own > 0 && lo <= x && x < lo + own) {
        *start_q = q0 + lane;
        start_x[2] = x - lo;
      }
      before += __shfl_sync(0xffffffffu, run, 31);
    }
  }
  fence_async_smem();  // the costs are read; TMA writes there next
  tc_fence_before();
  block_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  Walk<NS, BN> walk;
  walk.start(p, start_x[0], start_x[1], start_x[0] < start_x[1] ? *start_q : 0, start_x[2]);
  Segment s;
  bool ok = true;
  // A wait that ran out, or was told to stop, ends the CTA: every role goes
  // on through its loops without waiting or touching anything.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!ok) return;
    if (!mbar_wait(bar, parity, abort_flag)) {
      if (!*abort_flag) report(p.status, MFD_ERR_TIMEOUT);
      *abort_flag = 1;
      ok = false;
    }
  };
  // The order in which a segment's tiles pass the ring: keys and values of
  // tile j as K0 V0 K1 V1 .. when both streams read every tile, K0 K1 V0 K2 V1 ..
  // when they take turns (a stream's scores are then two tiles ahead).  Step i
  // of 2 n: returns the tile, negative (-1 - tile) for values.
  auto order = [](int n, bool shared, int i) {
    if (shared || n == 1) return (i & 1) ? -1 - (i >> 1) : i >> 1;
    if (i == 0) return 0;
    if (i == 2 * n - 1) return -1 - (n - 1);
    return (i & 1) ? (i + 1) >> 1 : -1 - ((i - 2) >> 1);
  };

  if (warp < 4) {
    if (NS == 2) regs_down<64>();
    if (warp == 0) {
      // ------------------------------------------------------- loads
      // Keys and values of one token serve M rows of this CTA only, or of
      // neighbours too when there are more row tiles: then they stay in L2.
      const uint64_t policy = p.n_pair > 1 ? policy_evict_normal() : policy_evict_first();
      const int ps = 1 << cv.ps_shift;
      const int rows = ps < BN ? ps : BN;  // of a box
          uint32_t n = 0, special_par = 0, issued = 0, issued_special = 0, issued_par = 0;
      while (walk.next(p, s)) {
        const int nt = s.t1 - s.t0;
        const bool shared = s.it.active == 2;
        const int len = s.ctx + s.nn;
        for (int i = 0; i < 2 * nt; ++i) {
          const int o = order(nt, shared, i);
          const bool is_v = o < 0;
          const int base = (s.t0 + (is_v ? -1 - o : o)) * BN;
          // boxes with positions before the end
          const int some = (min(len - base, BN) + rows - 1) / rows;
          int page = 0;
          if (lane < some) {
            page = __ldg(cv.table + (size_t)s.q * cv.max_pages + ((base + lane * rows) >> cv.ps_shift));
            if (page < 0 || page >= cv.n_pages) {
              report(p.status, MFD_ERR_INPUT);
              page = cv.n_pages;  // outside the map: reads as zeros
            }
          }
          if (E4M3) {
            const int st = (int)(n % RN);
            wait(&raw_empty[st], ((n / RN) & 1u) ^ 1u);
            if (__all_sync(0xffffffffu, ok)) {
              if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], (uint32_t)(some * rows * cv.D));
              __syncwarp();
              if (lane < some)
                tma_load_4d(sR + st * SH::RAW + lane * rows * cv.D, is_v ? &map_v : &map_k, 0,
                            (base + lane * rows) & (ps - 1), s.h, page, &raw_full[st], policy);
              issued |= 1u << st;
              const uint32_t par = (n / RN) & 1u;
              issued_par = (issued_par & ~(1u << st)) | (par << st);
            }
          } else {
            const int st = (int)(n % ST);
            wait(&empty[st], ((n / ST) & 1u) ^ 1u);
            const bool sp = is_v && base + BN > s.ctx;
            uint64_t *bar = sp ? &special[st] : &full[st];
            if (__all_sync(0xffffffffu, ok)) {
              if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(some * rows * 128 * NB));
              __syncwarp();
              if (lane < some)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                  tma_load_4d(sT + st * SH::STAGE + b * (BN * 128) + lane * rows * 128, is_v ? &map_v : &map_k, b * 64,
                              (base + lane * rows) & (ps - 1), s.h, page, bar, policy);
              issued |= 1u << st;
              const uint32_t par = sp ? (special_par >> st) & 1u : (n / ST) & 1u;
              issued_par = (issued_par & ~(1u << st)) | (par << st);
              issued_special = (issued_special & ~(1u << st)) | ((sp ? 1u : 0u) << st);
              if (sp) special_par ^= 1u << st;
            }
          }
          ++n;
        }
      }
      // every load issued lands before the CTA may exit
      if (lane == 0)
        for (int st = 0; st < (E4M3 ? RST : ST); ++st)
          if ((issued >> st) & 1u)
            mbar_wait(E4M3 ? &raw_full[st] : ((issued_special >> st) & 1u) ? &special[st] : &full[st],
                      (issued_par >> st) & 1u, never);
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        // ----------------------------------------------------- MMAs
        constexpr uint32_t id_s = idesc_16<T>(BM, BN, false), id_o = idesc_16<T>(BM, DP, true);
        const int k_steps = (cv.D + 15) / 16;
        uint32_t n = 0;  // ring position
        uint32_t seg = 0, p_par = 0;
        while (walk.next(p, s)) {
          const int nt = s.t1 - s.t0;
          if (nt == 0) continue;
          const bool shared = s.it.active == 2;
          const int steps = shared ? 2 * nt : nt;
          wait(q_full, seg & 1u);
          ++seg;
          uint32_t kst = 0, vst = 0;
          auto scores = [&](int i) {
            if (!shared || !(i & 1)) {
              kst = n % ST;
              wait(&full[kst], (n / ST) & 1u);
              ++n;
            }
            if (!ok) return;
            tc_fence_after();
            const uint32_t qa = smem_u32(sQ) + (shared ? (uint32_t)(i & 1) * SH::Q_TILE : 0u);
            const uint32_t ka = smem_u32(sT) + kst * SH::STAGE;
            const uint32_t d = tmem + SH::TM_S + (uint32_t)(i & 1) * BN;
            for (int k = 0; k < k_steps; ++k) {
              const uint64_t ad = smem_desc_sw128(qa + (uint32_t)(k >> 2) * (BM * 128) + (uint32_t)(k & 3) * 32);
              const uint64_t bd = smem_desc_sw128(ka + (uint32_t)(k >> 2) * (BN * 128) + (uint32_t)(k & 3) * 32);
              tc_mma_f16(d, ad, bd, id_s, k != 0);
            }
            tc_commit(&s_full[i & 1]);
            if (!shared || (i & 1)) tc_commit(&empty[kst]);
          };
          auto values = [&](int i) {
            wait(&p_full[i & 1], (p_par >> (i & 1)) & 1u);
            p_par ^= 1u << (i & 1);
            if (!shared || !(i & 1)) {
              vst = n % ST;
              wait(&full[vst], (n / ST) & 1u);
              ++n;
            }
            if (!ok) return;
            tc_fence_after();
            const int acc = NS == 2 ? i & 1 : 0;
            const uint32_t va = smem_u32(sT) + vst * SH::STAGE;
            const uint32_t d = tmem + SH::TM_O + (uint32_t)acc * DP;
            const uint32_t a = tmem + SH::TM_S + (uint32_t)(i & 1) * BN;
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              tc_mma_f16_ta(d, a + k * 8, smem_desc_sw128_mn(va + k * 2048, BN * 128), id_o,
                            (NS == 2 ? i >= 2 : i >= 1) || k != 0);
            tc_commit(&pv_done[acc]);
            if (!shared || (i & 1)) tc_commit(&empty[vst]);
          };
          scores(0);
          if (steps > 1) scores(1);
          for (int i = 0; i < steps; ++i) {
            values(i);
            if (i + 2 < steps) scores(i + 2);
          }
        }
        tc_commit(drain);  // all MMAs finish before tensor memory is released
        mbar_wait(drain, 0, never);
      }
      __syncwarp();
    }
  } else if (warp < SH::HELP_WARP) {
    // --------------------------------------------------------- softmax
    if (NS == 2) regs_up<192>();
    const int ws = NS == 2 ? (warp - 4) >> 2 : 0;  // stream
    const int wq = warp & 3;                       // the warp's lanes of tensor memory
    const int r = wq * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    uint32_t s_par = 0, pv_n = 0;
    // alternating streams exchange (m, l) in the space of the second Q tile
    float2 *ml_s = reinterpret_cast<float2 *>(sQ + (NS - 1) * SH::Q_TILE);
    while (walk.next(p, s)) {
      const int nt = s.t1 - s.t0;
      const bool shared = s.it.active == 2;
      const int live = s.nn * p.G;
      const int rt = shared ? ws : 0;                     // row tile of the group
      const int row = (s.pair * NS + rt) * BM + r;        // this thread's row
      const int node = row / p.G, g = row - node * p.G;
      const bool row_live = row < live && nt > 0;
      const bool warp_live = (s.pair * NS + rt) * BM + wq * 32 < live && nt > 0;

      // rows past n_nodes, once per item
      if (s.head) {
        const int zrow = (s.pair * NS + ws) * BM + r;
        if (zrow < p.M && zrow >= (s.it.tiles ? live : 0)) {
          const int zn = zrow / p.G, zg = zrow - zn * p.G;
          const int64_t at = ((int64_t)s.q * p.N + zn) * p.Hq + s.h * p.G + zg;
          for (int d = 0; d < cv.D; d += 8) *reinterpret_cast<uint4 *>(p.out + at * cv.D + d) = make_uint4(0, 0, 0, 0);
          if (p.lse) p.lse[at] = -INFINITY;
        }
      }
      if (nt == 0) continue;

      // queries: 16-byte chunks to the swizzled tile; rows that are not live
      // stay as they are (a row's scores reach no other row)
      {
        constexpr int C = DP / 8;
        const int tiles_rows = shared || NS == 1 ? BM : BM / 2;  // alternating: half the rows each
        const int row_first = shared || NS == 1 ? 0 : ws * (BM / 2);
        uint8_t *dst = sQ + rt * SH::Q_TILE;
        const int t128 = wq * 32 + lane;
        const int ch = t128 % C;
        for (int i = t128 / C; i < tiles_rows; i += 128 / C) {
          const int rr = row_first + i, grow = (s.pair * NS + rt) * BM + rr;
          if (grow >= live) break;
          const int n1 = grow / p.G, g1 = grow - n1 * p.G;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (ch * 8 < cv.D)
            x = __ldg(reinterpret_cast<const uint4 *>(p.q + ((int64_t)s.q * p.N + n1) * p.q_stride +
                                                      (int64_t)(s.h * p.G + g1) * cv.D + ch * 8));
          *reinterpret_cast<uint4 *>(dst + (ch >> 3) * (BM * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = x;
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);

      const int steps = shared ? 2 * nt : nt;
      const uint32_t *mask_row =
          p.mask && row_live ? p.mask + ((int64_t)s.q * p.N + node) * p.W32 : nullptr;
      float m = -INFINITY, l = 0.f;
      int done = 0;  // products with values of this stream's accumulator
      for (int i = NS == 2 ? ws : 0; i < steps; i += NS) {
        const int slot = i & 1;
        const int t_base = (s.t0 + (shared ? i >> 1 : i)) * BN;
        uint32_t vis[BN / 32];
        const bool edge = t_base + BN > s.ctx;
        if (edge && warp_live) {
#pragma unroll
          for (int k = 0; k < BN / 32; ++k)
            vis[k] = row_live ? visible32(mask_row, p.W32, node, s.nn, t_base + 32 * k - s.ctx) : 0u;
        }
        wait(&s_full[slot], (s_par >> slot) & 1u);
        s_par ^= 1u << slot;
        ok = __all_sync(0xffffffffu, ok);
        if (ok && warp_live) {
          tc_fence_after();
          const uint32_t sa = lane_base + SH::TM_S + (uint32_t)slot * BN;
          uint32_t xr[BN];
#pragma unroll
          for (int k = 0; k < BN / 32; ++k) tmem_ld32(sa + 32 * k, xr + 32 * k);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < BN / 32; ++k) tie32(xr + 32 * k);
          if (edge) {
#pragma unroll
            for (int k = 0; k < BN; ++k) xr[k] = (vis[k >> 5] >> (k & 31)) & 1u ? xr[k] : 0xFF800000u;
          }
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = __uint_as_float(xr[k]);
#pragma unroll
          for (int k = 4; k < BN; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(xr[k]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
          // move the maximum when it has grown by enough (or is the first)
          const bool move = row_live && top > m + MAX_GROWTH;
          if (__any_sync(0xffffffffu, move)) {
            const float m2 = move ? top : m;
            const float a = move ? ex2(m - m2) : 1.f;
            m = m2;
            l *= a;
            if (done) {
              wait(&pv_done[ws], (pv_n - 1u) & 1u);
              tc_fence_after();
              const uint32_t oa = lane_base + SH::TM_O + (uint32_t)ws * DP;
#pragma unroll 1
              for (int d = 0; d < DP; d += 16) {
                uint32_t o[16];
                tmem_ld16(oa + d, o);
                tmem_wait_ld();
                tie16(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                tmem_st16(oa + d, o);
              }
            }
          }
          const float mz = m == -INFINITY ? 0.f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int part = 0; part < BN / 32; ++part) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float a = ex2(fmaf(__uint_as_float(xr[32 * part + 2 * k]), p.c, -mz));
              const float b = ex2(fmaf(__uint_as_float(xr[32 * part + 2 * k + 1]), p.c, -mz));
              sum[(2 * k) & 3] += a;
              sum[(2 * k + 1) & 3] += b;
              pk[k] = pack2<T>(a, b);
            }
            tmem_st16(sa + 16 * part, pk);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&p_full[slot]);
        ++done;
        ++pv_n;
      }

      // ------------------------------------------------------- epilogue
      // With one stream the last but one product may still run (scores are two
      // tiles ahead of it); a wait on a parity needs the phase before it complete.
      if (NS == 1 && done > 1) wait(&pv_done[ws], pv_n & 1u);
      if (done) wait(&pv_done[ws], (pv_n - 1u) & 1u);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const bool alternating = NS == 2 && !shared;
      float a0 = 1.f, a1 = 0.f;
      if (alternating) {
        if (ws == 1) ml_s[r] = make_float2(m, l);
        named_sync(1, 256);
        if (ws == 0) {
          const float2 o = ml_s[r];
          const float top = fmaxf(m, o.x);
          if (top > -INFINITY) {
            a0 = m == -INFINITY ? 0.f : ex2(m - top);
            a1 = o.x == -INFINITY ? 0.f : ex2(o.x - top);
            l = l * a0 + o.y * a1;
            m = top;
          } else {
            l += o.y;  // nothing seen (0), or NaN
          }
        }
      }
      const bool whole = s.t0 == 0 && s.t1 == s.it.tiles;
      if (ok && (!alternating || ws == 0) && warp_live) {
        const bool two = alternating && steps > 1;
        const uint32_t oa = lane_base + SH::TM_O + (uint32_t)(alternating ? 0 : ws) * DP;
        const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        const int64_t at = row_live ? ((int64_t)s.q * p.N + node) * p.Hq + s.h * p.G + g : 0;
        const int prow = rt * BM + r;
        const int slot = 2 * (int)blockIdx.x + (s.t0 == 0 ? 1 : 0);
        const bool fix = p.N > 1 && s.t1 * BN > s.ctx && *any_bad;
        // the values' place, for those added back
        const int hstart = s.h;
#pragma unroll 1
        for (int d = 0; d < DP; d += 32) {
          if (d >= cv.D) break;
          uint32_t o[32], o1[32];
          tmem_ld32(oa + d, o);
          if (two) tmem_ld32(oa + DP + d, o1);
          tmem_wait_ld();
          tie32(o);
          if (two) tie32(o1);
          float f[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float x = __uint_as_float(o[k]);
            if (alternating) {
              x *= a0;
              if (two) x = fmaf(__uint_as_float(o1[k]), a1, x);
            }
            f[k] = x * inv;
          }
          if (fix && row_live) {
            const int lo = max(0, s.t0 * BN - s.ctx), hi = min(s.nn, s.t1 * BN - s.ctx);
            for (int j = lo; j < hi; ++j) {
              if (!((bad[j >> 5] >> (j & 31)) & 1u)) continue;
              const bool sees = mask_row ? (__ldg(mask_row + (j >> 5)) >> (j & 31)) & 1u : j <= node;
              if (!sees) continue;
              const int pos = s.ctx + j;
              const int page = __ldg(cv.table + (size_t)s.q * cv.max_pages + (pos >> cv.ps_shift));
              if (page < 0 || page >= cv.n_pages) continue;
              const int64_t e = page * cv.page_stride + hstart * cv.head_stride +
                                (int64_t)(pos & ((1 << cv.ps_shift) - 1)) * cv.token_stride;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                if (d + k < cv.D) {
                  if (E4M3) {
                    f[k] = __int_as_float(0x7FFFFFFF);
                  } else {
                    const uint32_t w = static_cast<const uint16_t *>(cv.v)[e + d + k];
                    if (nonfinite2<T>(w)) f[k] += unpack2<T>(w).x;
                  }
                }
              }
            }
          }
          if (row_live) {
            if (whole) {
#pragma unroll
              for (int k = 0; k < 32; k += 8)
                if (d + k < cv.D) {
                  float y[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e) y[e] = f[k + e];
                  *reinterpret_cast<uint4 *>(p.out + at * cv.D + d + k) = pack8<T>(y);
                }
            } else {
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                if (d + k < cv.D)
                  p.part_o[((int64_t)slot * (cv.D / 4) + (d + k) / 4) * p.part_rows + prow] =
                      make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
            }
          }
        }
        if (row_live) {
          if (whole) {
            if (p.lse) p.lse[at] = m == -INFINITY && l == 0.f ? -INFINITY : m * LN2 + logf(l);
          } else {
            p.part_ml[(int64_t)slot * p.part_rows + prow] = make_float2(m, l);
          }
        }
      }
      tc_fence_before();
      if (alternating) named_sync(1, 256);  // the first stream has read the second's O and (m, l)
      tc_fence_after();
      if (ws == 0)
        named_sync(2, 128);
      else
        named_sync(3, 128);
      if (r == 0) {
        __threadfence_block();
        seg_done[ws] = seg_done[ws] + 1;
      }
    }
  } else {
    // --------------------------------------------------------- helpers
    if (NS == 2) regs_down<64>();
    const int ht = tid - SH::HELP_WARP * 32;
    uint32_t n = 0, special_par = 0;
    int seg = 0;
    while (walk.next(p, s)) {
      const int nt = s.t1 - s.t0;
      if (nt == 0) continue;
      const bool shared = s.it.active == 2;
      const int len = s.ctx + s.nn;
      // one row per request: every key before the end is seen
      const bool note = p.N > 1;
      bool clean = false;  // the bad-node bits are this segment's
      // exponent bytes of position t (keys, values)
      auto codes = [&](int t, int &ck, int &cvv) {
        ck = cvv = 0;
        if (ht < BN && t < len) {
          const int page = __ldg(cv.table + (size_t)s.q * cv.max_pages + (t >> cv.ps_shift));
          if (page >= 0 && page < cv.n_pages) {
            const int64_t e = (((int64_t)page * cv.Hk + s.h) << cv.ps_shift) + (t & ((1 << cv.ps_shift) - 1));
            ck = __ldg(cv.k_exp + e);
            cvv = __ldg(cv.v_exp + e);
          }
        }
      };
      auto put_codes = [&](int j, int ck, int cvv) {
        if (ht < BN) {
          sC[(j & 7) * 128 + ht] = (uint8_t)ck;
          sC[1024 + (j & 7) * 128 + ht] = (uint8_t)cvv;
        }
      };
      if (E4M3) {
        named_sync(4, 128);  // every helper is done with the last segment's bytes
        int ck0, cv0, ck1, cv1;
        codes(s.t0 * BN + ht, ck0, cv0);
        codes((s.t0 + 1) * BN + ht, ck1, cv1);
        put_codes(0, ck0, cv0);
        put_codes(1, ck1, cv1);
      }
      for (int i = 0; i < 2 * nt; ++i) {
        const int o = order(nt, shared, i);
        const bool is_v = o < 0;
        const int j = is_v ? -1 - o : o;
        const int base = (s.t0 + j) * BN;
        const bool sp = is_v && base + BN > s.ctx;
        if (sp && note && !clean) {
          // the bits still serve the previous segment until its rows are out
          if (ok) {
            const unsigned long long t0 = globaltimer();
            for (uint32_t it = 1;; ++it) {
              if (seg_done[0] >= seg && (NS == 1 || seg_done[1] >= seg)) break;
              if ((it & 15u) == 0 && (*abort_flag || globaltimer() - t0 > kWaitLimitNs)) {
                if (!*abort_flag) report(p.status, MFD_ERR_TIMEOUT);
                *abort_flag = 1;
                ok = false;
                break;
              }
              __nanosleep(64);
            }
          }
          named_sync(4, 128);
          for (int k = ht; k < MAX_N / 32; k += 128) bad[k] = 0;
          if (ht == 0) *any_bad = 0;
          named_sync(4, 128);
          clean = true;
        }
        const int st = (int)(n % ST);
        if (E4M3) {
          const int rs = (int)(n % RN);
          int ck = 0, cvv = 0;
          if (!is_v) {
            named_sync(4, 128);  // this tile's exponent bytes are written
            if (j + 2 < nt) codes(base + 2 * BN + ht, ck, cvv);
          }
          wait(&empty[st], ((n / ST) & 1u) ^ 1u);
          wait(&raw_full[rs], (n / RN) & 1u);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            const uint8_t *src = sR + rs * SH::RAW;
            uint8_t *dst = sT + st * SH::STAGE;
            const uint8_t *code = sC + (is_v ? 1024 : 0) + (j & 7) * 128;
            constexpr int C = DP / 16;
#pragma unroll 4
            for (int k = 0; k < BN * C / 128; ++k) {
              const int idx = ht + 128 * k;
              const int tok = idx / C, ch = idx % C;
              uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
              const int t = base + tok;
              if (ch * 16 < cv.D && t < len) {
                const int cd = code[tok];
                if (cd != EXP_NAN) {
                  const uint4 x = *reinterpret_cast<const uint4 *>(src + tok * cv.D + ch * 16);
                  const Widen<T> widen(cd);
                  uint2 a = widen(x.x), b = widen(x.y);
                  lo = make_uint4(a.x, a.y, b.x, b.y);
                  a = widen(x.z);
                  b = widen(x.w);
                  hi = make_uint4(a.x, a.y, b.x, b.y);
                } else if (sp && note && t >= s.ctx) {
                  atomicOr(&bad[(t - s.ctx) >> 5], 1u << ((t - s.ctx) & 31));
                  *any_bad = 1;
                } else {
                  lo = hi = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
                }
              }
              uint8_t *row = dst + (ch >> 2) * (BN * 128) + tok * 128;
              const int c2 = (ch & 3) * 2, x7 = tok & 7;
              // neighbouring blocks' lanes write their two chunks in opposite order (other banks)
              const bool sw = (ch >> 2) & 1;
              *reinterpret_cast<uint4 *>(row + (((c2 + (sw ? 1 : 0)) ^ x7) << 4)) = sw ? hi : lo;
              *reinterpret_cast<uint4 *>(row + (((c2 + (sw ? 0 : 1)) ^ x7) << 4)) = sw ? lo : hi;
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0 && ok) {
            mbar_arrive(&raw_empty[rs]);
            mbar_arrive(&full[st]);
          }
          if (!is_v && j + 2 < nt) put_codes(j + 2, ck, cvv);
        } else if (sp) {
          wait(&special[st], (special_par >> st) & 1u);
          special_par ^= 1u << st;
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            uint8_t *dst = sT + st * SH::STAGE;
            constexpr int C = DP / 8;
#pragma unroll 4
            for (int k = 0; k < BN * C / 128; ++k) {
              const int idx = ht + 128 * k;
              const int tok = idx / C, ch = idx % C;
              const int t = base + tok;
              uint4 *at = reinterpret_cast<uint4 *>(dst + (ch >> 3) * (BN * 128) + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
              if (t >= len) {
                *at = make_uint4(0, 0, 0, 0);
              } else if (note && t >= s.ctx) {
                uint4 x = *at;
                if (nonfinite2<T>(x.x) | nonfinite2<T>(x.y) | nonfinite2<T>(x.z) | nonfinite2<T>(x.w)) {
                  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t z = nonfinite2<T>(w[e]);
                    if (z & 0x8000u) w[e] &= 0xFFFF0000u;
                    if (z & 0x80000000u) w[e] &= 0x0000FFFFu;
                  }
                  *at = make_uint4(w[0], w[1], w[2], w[3]);
                  atomicOr(&bad[(t - s.ctx) >> 5], 1u << ((t - s.ctx) & 31));
                  *any_bad = 1;
                }
              }
            }
          }
          fence_async_smem();
          named_sync(4, 128);
          if (ht == 0 && ok) mbar_arrive(&full[st]);
        }
        ++n;
      }
      ++seg;
    }
  }
  tc_fence_before();
  block_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join

// Combines the parts of an item that borders cut: one block per (pair of an
// item, request and head), a thread per row and 8 columns.
template <typename T, int NS, int BN>
__global__ void __launch_bounds__(256) join_kernel(const Params p, int n_cta) {
  __shared__ int64_t sums[2];  // before this request, in all
  const int pair = blockIdx.x, h = blockIdx.y, q = blockIdx.z, tid = threadIdx.x;
  if (tid < 2) sums[tid] = 0;
  block_sync();
  int64_t before = 0, total = 0;
  for (int i = tid; i < p.n_req; i += 256) {
    int ctx, nn;
    lengths(p, i, ctx, nn);
    const int64_t c = p.cv.Hk * head_cost<NS, BN>(p, ctx, nn);
    total += c;
    if (i < q) before += c;
  }
  if (total) atomicAdd(reinterpret_cast<unsigned long long *>(&sums[1]), (unsigned long long)total);
  if (before) atomicAdd(reinterpret_cast<unsigned long long *>(&sums[0]), (unsigned long long)before);
  block_sync();
  total = sums[1];
  int ctx, nn;
  lengths(p, q, ctx, nn);
  const Item it = item_of<NS, BN>(p, ctx, nn, pair);
  if (it.tiles == 0) return;
  int64_t u0 = sums[0] + h * head_cost<NS, BN>(p, ctx, nn);
  for (int i = 0; i < pair; ++i) u0 += item_of<NS, BN>(p, ctx, nn, i).cost;
  const int64_t u1 = u0 + it.cost;
  const int c0 = cta_of(total, u0, n_cta), c1 = cta_of(total, u1 - 1, n_cta);
  if (c0 == c1) return;
  // a part's key tiles; returns its slot, or -1 if it holds none, -2 if all
  auto slot_of = [&](int c) {
    const int64_t lo = border(total, c, n_cta), hi = border(total, c + 1, n_cta);
    const int a = (int)((lo > u0 ? lo : u0) - u0), b = (int)((hi < u1 ? hi : u1) - u0);
    const int t0 = tile_at(it, a), t1 = tile_at(it, b);
    if (t0 >= t1) return -1;
    if (t0 == 0 && t1 == it.tiles) return -2;
    return 2 * c + (t0 == 0 ? 1 : 0);
  };
  const int first = pair * NS * BM;
  const int rows = min(nn * p.G - first, NS * BM);
  const int C8 = p.cv.D / 8;
  for (int i = tid; i < rows * C8; i += 256) {
    const int r = i % rows, ch = i / rows;
    float m = -INFINITY, l = 0.f, acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    bool direct = false;
    for (int c = c0; c <= c1; ++c) {
      const int s = slot_of(c);
      if (s == -1) continue;
      if (s == -2) {
        direct = true;
        break;
      }
      const float2 ml = p.part_ml[(int64_t)s * p.part_rows + r];
      const float4 a = p.part_o[((int64_t)s * (p.cv.D / 4) + 2 * ch) * p.part_rows + r];
      const float4 b = p.part_o[((int64_t)s * (p.cv.D / 4) + 2 * ch + 1) * p.part_rows + r];
      const float top = fmaxf(m, ml.x);
      const float w0 = m == -INFINITY ? 0.f : ex2(m - top), w1 = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
      const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      if (ml.x == -INFINITY && ml.y == 0.f) continue;  // this part's keys are not seen
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = (m == -INFINITY ? 0.f : acc[k] * w0) + x[k] * w1;
      l = l * w0 + (ml.x == -INFINITY ? ml.y : ml.y * w1);
      m = top;
    }
    if (direct) return;
    const int node = (first + r) / p.G, g = first + r - node * p.G;
    const int64_t at = ((int64_t)q * p.N + node) * p.Hq + h * p.G + g;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = acc[k] * inv;
    *reinterpret_cast<uint4 *>(p.out + at * p.cv.D + ch * 8) = pack8<T>(y);
    if (p.lse && ch == 0) p.lse[at] = m == -INFINITY && l == 0.f ? -INFINITY : m * LN2 + logf(l);
  }
}

template <typename T, int DP, bool E4M3>
cudaError_t launch_shape(const AttentionLaunch &A, const Params &p, int n_cta, cudaStream_t stream) {
  using SH = Shape<DP, E4M3>;
  static_assert(SH::SMEM <= 232448, "shared memory of one CTA");
  cudaError_t e = cudaFuncSetAttribute(attention_kernel<T, DP, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::SMEM);
  if (e != cudaSuccess) return e;
  attention_kernel<T, DP, E4M3><<<n_cta, SH::THREADS, SH::SMEM, stream>>>(*A.map_k, *A.map_v, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  join_kernel<T, SH::NS, SH::BN><<<dim3(p.n_pair, p.cv.Hk, p.n_req), 256, 0, stream>>>(p, n_cta);
  return cudaGetLastError();
}

template <typename T, bool E4M3>
cudaError_t launch_width(const AttentionLaunch &A, const Params &p, int n_cta, cudaStream_t stream) {
  if (A.cache.D <= 64) return launch_shape<T, 64, E4M3>(A, p, n_cta, stream);
  if (A.cache.D <= 128) return launch_shape<T, 128, E4M3>(A, p, n_cta, stream);
  return launch_shape<T, 256, E4M3>(A, p, n_cta, stream);
}

int row_group(int D) { return (D > 128 ? 1 : 2) * BM; }
int part_rows(int M, int D) { return M < row_group(D) ? (M + 7) / 8 * 8 : row_group(D); }

}  // namespace

size_t attention_part_bytes(int M, int D) {
  // two parts at most for every CTA: of the item its stretch starts in, and of the one it ends in
  return (size_t)2 * ATTENTION_MAX_CTAS * part_rows(M, D) * ((size_t)D * 4 + 8);
}
int attention_box_rows(int page_size, int D) {
  const int bn = D > 128 ? 64 : 128;
  return page_size < bn ? page_size : bn;
}

cudaError_t launch_tree_attention(const AttentionLaunch &A, cudaStream_t stream) {
  Params p;
  p.cv = A.cache;
  p.q = static_cast<const uint16_t *>(A.q);
  p.q_stride = A.q_stride;
  p.n_req = A.n_req;
  p.N = A.N;
  p.Hq = A.Hq;
  p.G = A.Hq / A.cache.Hk;
  p.M = A.N * p.G;
  p.W32 = (A.N + 31) / 32;
  p.n_pair = (p.M + row_group(A.cache.D) - 1) / row_group(A.cache.D);
  p.ctx_len = A.ctx_len;
  p.n_nodes = A.n_nodes;
  p.mask = A.mask;
  p.c = A.scale * LOG2E;
  p.out = static_cast<uint16_t *>(A.out);
  p.lse = A.lse;
  p.status = A.status;
  p.part_rows = part_rows(p.M, A.cache.D);
  p.part_o = static_cast<float4 *>(A.ws);
  p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(A.ws) +
                                         (size_t)2 * ATTENTION_MAX_CTAS * p.part_rows * A.cache.D * 4);
  const int n_cta = A.n_sm < ATTENTION_MAX_CTAS ? A.n_sm : ATTENTION_MAX_CTAS;
  const bool e4m3 = A.cache.dtype == MFD_E4M3;
  if (A.dtype == MFD_BF16)
    return e4m3 ? launch_width<__nv_bfloat16, true>(A, p, n_cta, stream)
                : launch_width<__nv_bfloat16, false>(A, p, n_cta, stream);
  return e4m3 ? launch_width<__half, true>(A, p, n_cta, stream) : launch_width<__half, false>(A, p, n_cta, stream);
}

}  // namespace mfd
