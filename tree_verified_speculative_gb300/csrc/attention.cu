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
// one stream, with two S accumulators used in turn; a 16-bit cache's has two
// softmax warpgroups, each with half of a row's columns (an 8-bit cache's
// helpers leave no room for the second).
//
// Work split.  All (request, key head, row tile pair) items and their key
// tiles form one line, ordered so that the row tiles of a head, which read
// the same keys, are neighbours; every CTA takes an equal stretch of it.  An
// item cut by a border leaves its parts (O, m, l) in scratch, and join_kernel
// combines them in a fixed order.  The line is laid out from the lengths on
// the device: a short and a long request keep all SMs busy alike, and a graph
// replays with other lengths.
//
// Warps: 0 loads keys and 3 values (TMA, one box per page and 64 columns), 1
// issues the MMAs, 2 makes the list of work and turns E4M3 rows' exponent bytes
// into powers, then the softmax warpgroups, then the helpers: two warpgroups
// that widen E4M3 tiles to the operand type, or one that goes over value tiles
// of 16-bit caches that reach past the context.  There it clears rows past the
// end and values that are not finite, which a product would spread to rows that
// do not see them (0 * NaN); a cleared value's node is noted and added back for
// the rows that do see it.  E4M3 rows that read back as NaN, or past the type's
// range, are taken out and added back the same way.
//
// What bounds it, on the GPU alone (a captured call replayed):
//   one token over 200,002 positions, 32/8 heads of 128, bf16: HBM; 129 us, 6.4
//     TB/s, 0.94 of what a copy reaches
//   32 requests of one token over ragged contexts up to 16,000, the same heads,
//     E4M3: the widening; 236 us, 3.2 TB/s, each byte read being one
//     element to turn into two bytes (one helper warpgroup instead of two: 297)
//   32 trees of 129 nodes over up to 6,000, the same heads, E4M3: a stream's
//     chain of scores, softmax and product; 403 us, 0.69 PFLOP/s (16-bit: 346).  A step of 128
//     rows and 128 keys takes 2,900 cycles of which the tensor pipe needs 1,024;
//     neither issue slots (51 %) nor exponentials (16 %) are used up
//   one tree of 257 nodes over 8,191, 16/4 heads of 256, bf16: 61 us; of that
//     the pipelines' filling, the cut items' parts (20 MB) and their join take
//     half, the products 0.57 PFLOP/s over the whole
//   three prompts of 1,777 tokens, 28/4 heads of 80, fp16: 131 us, the same
//     chain, and starts and ends of items of ten tiles
#include <atomic>
#include <climits>

#include "join_note.h"
#include "kvcache.h"
#include "mfd_device.cuh"

namespace mfd {
namespace {

constexpr int BM = 128;  // rows of a tile
constexpr int BN = 128;  // key positions of a tile
constexpr int MAX_N = 4096;
constexpr int SEG_RING = 4;  // entries of a CTA's list of work in flight
constexpr float LN2 = 0.6931471805599453f;
// What an item's start and end cost, in steps: the queries' load, the pipeline's
// filling and draining, the output.  Measured with 1, 4, 5 and 6: three prompts of
// 1,777 rows 152, 131, 131, 135 us; 32 trees of 129 nodes 410, 400, 402, 397; one
// tree of 257 nodes 59.5, 60.8, 60.9, 60.9.
constexpr int START_COST = 5;
constexpr float LARGE_SCORE = 65536.f;
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
  Cut *cuts;  // [CTA]
};

template <int DP_, bool E4M3_>
struct Shape {
  static constexpr int DP = DP_;                       // head width, padded to 64, 128 or 256
  static constexpr int NS = DP == 256 ? 1 : 2;         // streams
  static constexpr int UC = DP == 64 ? 64 : 128;       // columns of a unit, what one stage holds of a tile
  static constexpr int NU = DP / UC;                   // units of a tile
  static constexpr int NB = UC / 64;                   // 64-column blocks of 128-byte rows
  static constexpr int Q_TILE = BM * DP * 2;
  static constexpr int STAGE = BN * UC * 2;
  static constexpr int RAW = BN * UC;                  // an E4M3 unit as it is in the cache
  static constexpr int ST = E4M3_ ? (DP == 64 ? 4 : 3) : (DP == 64 ? 8 : 5);
  static constexpr int RST = E4M3_ ? (DP == 64 ? 6 : 4) : 0;
  static constexpr int HELPERS = E4M3_ ? 2 : 1;        // warpgroups that help
  static constexpr bool SPLIT = NS == 1 && !E4M3_;     // one stream's columns shared by two softmax warpgroups
  static constexpr int SG = NS == 2 || SPLIT ? 2 : 1;  // softmax warpgroups
  static constexpr int THREADS = 128 * (1 + SG + HELPERS);
  static constexpr int HELP_WARP = 4 + 4 * SG;
  static constexpr int SW = 32;                        // score columns a softmax thread holds
  static constexpr int TM_S = 0;                       // two S accumulators; P over them
  static constexpr int TM_O = 2 * BN;
  static constexpr int POWERS = E4M3_ ? 2 * 4 * BN * 2 : 0;  // [k, v][tile mod 4][position], 16 bits
  static constexpr int BARS = (E4M3_ ? 2 : 3) * ST + 2 * RST + 8 + (E4M3_ ? 8 : 0) + 2 * SEG_RING;
  static constexpr int TOPS = SPLIT ? 2 * 2 * BM * 4 : 0;  // row maxima the two exchange, [step mod 2][half]
  static constexpr int SMEM = NS * Q_TILE + ST * STAGE + RST * RAW + POWERS + MAX_N / 8 + BARS * 8 + SEG_RING * 40 + 48 + TOPS;
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
  int cost;    // places on the line: a step per row tile and key tile, and START_COST (1 without live rows)
};

template <int NS>
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
  it.cost = it.active * it.tiles + (it.active ? START_COST : 1);
  return it;
}

// A key head's length on the line where it has one form for all of its items
// (a tree mask, or one item): by one thread.
template <int NS>
__device__ __forceinline__ int64_t head_cost(const Params &p, int ctx, int nn) {
  if (p.n_pair == 1) return item_of<NS>(p, ctx, nn, 0).cost;
  const int live = nn * p.G;
  const int pairs = (live + NS * BM - 1) / (NS * BM);  // with live rows
  return (int64_t)((live + BM - 1) / BM) * (nn ? (ctx + nn + BN - 1) / BN : 0) + p.n_pair + (int64_t)pairs * (START_COST - 1);
}
__device__ __forceinline__ bool one_form(const Params &p) { return p.mask || p.n_pair == 1; }
__device__ __forceinline__ int64_t warp_total(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int64_t warp_running(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}
// The same for any item lengths, by a warp, an item a lane at a time.
template <int NS>
__device__ __forceinline__ int64_t head_cost_warp(const Params &p, int ctx, int nn, int lane) {
  if (one_form(p)) return head_cost<NS>(p, ctx, nn);
  int64_t c = 0;
  for (int i = lane; i < p.n_pair; i += 32) c += item_of<NS>(p, ctx, nn, i).cost;
  return warp_total(c);
}
// The line's length (all requests), by a warp; with `x` also the request whose
// stretch holds place x and where that stretch starts.
template <int NS>
__device__ __forceinline__ int64_t line_walk(const Params &p, int lane, int64_t x, bool report_bad, int &q, int64_t &start) {
  int64_t total = 0;
  q = 0;
  start = 0;
  for (int b = 0; b < p.n_req; b += one_form(p) ? 32 : 1) {
    int ctx, nn;
    int64_t own = 0;
    if (one_form(p)) {
      if (b + lane < p.n_req) {
        if (!lengths(p, b + lane, ctx, nn) && report_bad) report(p.status, MFD_ERR_INPUT);
        own = p.cv.Hk * head_cost<NS>(p, ctx, nn);
      }
      if (x >= 0) {
        const int64_t run = total + warp_running(own, lane), lo = run - own;
        const unsigned hit = __ballot_sync(0xffffffffu, own > 0 && lo <= x && x < run);
        if (hit) {
          q = b + __ffs(hit) - 1;
          start = __shfl_sync(0xffffffffu, lo, __ffs(hit) - 1);
        }
        total = __shfl_sync(0xffffffffu, run, 31);
      } else {
        total += warp_total(own);
      }
    } else {
      if (!lengths(p, b, ctx, nn) && report_bad && lane == 0) report(p.status, MFD_ERR_INPUT);
      own = p.cv.Hk * head_cost_warp<NS>(p, ctx, nn, lane);
      if (x >= total && x < total + own) {
        q = b;
        start = total;
      }
      total += own;
    }
  }
  return total;
}
// The item of a head at `rest` places from the head's start, by a warp; `rest`
// becomes the place inside the item.
template <int NS>
__device__ __forceinline__ int find_item(const Params &p, int ctx, int nn, int lane, int64_t &rest) {
  if (p.n_pair == 1) return 0;
  for (int b = 0; b < p.n_pair; b += 32) {
    const int64_t own = b + lane < p.n_pair ? item_of<NS>(p, ctx, nn, b + lane).cost : 0;
    const int64_t run = warp_running(own, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, own > 0 && rest < run);
    if (hit) {
      const int l = __ffs(hit) - 1;
      rest -= __shfl_sync(0xffffffffu, run - own, l);
      return b + l;
    }
    rest -= __shfl_sync(0xffffffffu, run, 31);
  }
  return 0;  // not reached: rest lies inside the head
}

// Where the line's place x falls: CTA c of n has [C c / n, C (c + 1) / n).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {  // non-negative; mostly 32 bits
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t border(int64_t total, int c, int n) { return divide(total * c, n); }
__device__ __forceinline__ int cta_of(int64_t total, int64_t x, int n) { return (int)divide((x + 1) * n - 1, total); }

// First key tile at or after place z of an item.
__device__ __forceinline__ int tile_at(const Item &it, int z) {
  return z >= it.cost ? it.tiles : (int)divide((int64_t)z * it.tiles, it.cost);
}

// ------------------------------------------------------------------ primitives

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// 16 bytes global -> shared without a register; cp_async_wait waits for all of the thread's.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ void st_global16(void *dst, uint4 v) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// One lane of the warp; the branch it guards runs in uniform registers, which
// is where the MMA takes its operands from.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// Operand descriptors of 128-byte swizzled rows in shared memory (8-row groups
// 1024 bytes apart: stride byte offset; version 1; swizzle mode 128 bytes).
// Low word: address >> 4, and at bit 16 the leading byte offset >> 4: unused
// (1) where the contraction runs along the rows (queries, keys), the distance
// of 64-column blocks where it runs down them (values).
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead) { return (saddr >> 4) | ((lead >> 4) << 16); }

// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit operands, fp32 accumulate.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem].
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

// Whether some of eight elements are not finite, and the eight without those.
template <typename T>
__device__ __forceinline__ bool any_nonfinite(const uint4 &x) {
  return (nonfinite2<T>(x.x) | nonfinite2<T>(x.y) | nonfinite2<T>(x.z) | nonfinite2<T>(x.w)) != 0;
}
template <typename T>
__device__ __forceinline__ uint4 without_nonfinite(const uint4 &x) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t z = nonfinite2<T>(w[e]);
    if (z & 0x8000u) w[e] &= 0xFFFF0000u;
    if (z & 0x80000000u) w[e] &= 0x0000FFFFu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Notes that node j has values taken out.
__device__ __forceinline__ void note_node(int j, uint32_t *bad, volatile int *any_bad) {
  atomicOr(&bad[j >> 5], 1u << (j & 31));
  *any_bad = 1;
}

// E4M3 to the operand type.  A row's power is a 16-bit number that scales its
// values as widen4 takes them (NaN where the row reads back as NaN); `wide`
// says that the power has no such number and widen4_wide is to be used.  Four
// columns c0 .. c3 of a 32-bit word come out as (c1, c3), (c0, c2), which needs
// no byte permutation: the queries are put in the same order, and the output's
// columns are taken back from it.  The byte's exponent and mantissa bits are
// moved to the type's places, subnormals included, which reads as the value
// times 2^-120 in bf16 (biases 7 and 127) and 2^-8 in fp16 (7 and 15); one
// multiplication by a power of two puts both right.
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); }
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }
__device__ __forceinline__ uint32_t bits_of(__half2 v) { return *reinterpret_cast<const uint32_t *>(&v); }
template <typename T>
struct Widen;
template <>
struct Widen<__nv_bfloat16> {
  static __device__ __forceinline__ uint16_t power(int code, bool &wide) {
    if (code == EXP_NAN) return 0x7FFF;
    wide |= code > 134;
    return (uint16_t)((code > 134 ? 254 : code + 120) << 7);
  }
  static __device__ __forceinline__ uint2 widen4(uint32_t x, uint32_t power2) {
    const uint32_t hi = (x & 0x80008000u) | ((x >> 4) & 0x07F007F0u);
    const uint32_t lo = ((x * 256u) & 0x80008000u) | ((x * 16u) & 0x07F007F0u);
    return make_uint2(bits_of(__hmul2(as_bf162(hi), as_bf162(power2))), bits_of(__hmul2(as_bf162(lo), as_bf162(power2))));
  }
  // 2^(e + 120) in two multiplications
  static __device__ __forceinline__ uint2 widen4_wide(uint32_t x, int code) {
    const uint32_t rest = (uint32_t)(code - 7) << 7;
    const uint2 o = widen4(x, 0x7F007F00u);
    const __nv_bfloat162 f = as_bf162(rest | (rest << 16));
    return make_uint2(bits_of(__hmul2(as_bf162(o.x), f)), bits_of(__hmul2(as_bf162(o.y), f)));
  }
};
template <>
struct Widen<__half> {
  // 2^(e + 8) from 2^-24 (code 95) to 2^15; nothing of a row with code 0 is left in fp16
  static __device__ __forceinline__ uint16_t power(int code, bool &wide) {
    if (code == EXP_NAN) return 0x7FFF;
    wide |= (code > 0 && code < 95) || code > 134;
    return code == 0 ? 0 : code < 95 ? 1 : code < 105 ? (uint16_t)(1u << (code - 95)) : code > 134 ? 0x7800 : (uint16_t)((code - 104) << 10);
  }
  static __device__ __forceinline__ uint2 widen4(uint32_t x, uint32_t power2) {
    const uint32_t hi = (x & 0x80008000u) | ((x >> 1) & 0x3F803F80u);
    const uint32_t lo = ((x * 256u) & 0x80008000u) | ((x * 128u) & 0x3F803F80u);
    return make_uint2(bits_of(__hmul2(as_half2(hi), as_half2(power2))), bits_of(__hmul2(as_half2(lo), as_half2(power2))));
  }
  static __device__ __forceinline__ uint2 widen4_wide(uint32_t x, int code) {
    const float s = e4m3_scale(code);
    const float2 a = e4m3x2_float(x & 0xFFFFu), b = e4m3x2_float(x >> 16);
    return make_uint2(pack2<__half>(a.y * s, b.y * s), pack2<__half>(a.x * s, b.x * s));
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

// One entry of a CTA's list of work; q < 0 ends it.
struct Segment {
  int q, h, pair;
  int ctx, nn;
  int active, tiles;  // of the item
  int t0, t1;         // its key tiles in this stretch
  int head;           // the stretch has the item's start
};
// How long a role waits for its next entry: longer than the list's own waits,
// so that either every role gets an entry or none does.
constexpr unsigned long long SEG_LIMIT_NS = 4 * kWaitLimitNs;

// A waiting warp is put to sleep for up to a microsecond at a time: a dozen
// waiting warps that poll take the issue slots of those that work.
__device__ __forceinline__ bool try_wait_sleep(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
}
// Waits for the phase with `parity`; false when the limit passes or *abort is
// set.  Out of line, like all that is not taken for every tile: the roles' hot
// code shares an instruction cache that is small for it.
__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, unsigned long long limit_ns, volatile int *abort) {
  const unsigned long long t0 = globaltimer();
  for (;;) {
    if (try_wait_sleep(bar, parity)) return true;
    if (*abort || globaltimer() - t0 > limit_ns) return false;
  }
}
__device__ __forceinline__ bool wait_limit(uint64_t *bar, uint32_t parity, unsigned long long limit_ns,
                                           volatile int *abort) {
  return try_wait_sleep(bar, parity) || wait_long(bar, parity, limit_ns, abort);
}
// A pipeline wait that ran out, or was told to stop.
__device__ __noinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int32_t *status) {
  if (wait_long(bar, parity, kWaitLimitNs, abort_flag)) return true;
  if (!*abort_flag) report(status, MFD_ERR_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// Scores of a warp's rows that a tile past the context hides, to -infinity, in
// tensor memory: 32 columns per word of `vis`.
__device__ __noinline__ void hide_scores(uint32_t sa, int columns, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
#pragma unroll 1
  for (int part = 0; part < columns / 16; ++part) {
    const uint32_t w = (part < 2 ? v0 : part < 4 ? v1 : part < 6 ? v2 : v3) >> (16 * (part & 1));
    uint32_t x[16];
    tmem_ld16(sa + 16 * part, x);
    tmem_wait_ld();
    tie16(x);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = (w >> k) & 1u ? x[k] : 0xFF800000u;
    tmem_st16(sa + 16 * part, x);
  }
  tmem_wait_st();
}
// Scores so large that a product and a difference in one rounding would leave
// the maximum itself well off 2^0: each minus the maximum, rounded as the
// maximum was, in tensor memory.
__device__ __noinline__ void center_scores(uint32_t sa, int columns, float c, float m) {
  const float back = 1.f / c;
#pragma unroll 1
  for (int d = 0; d < columns; d += 16) {
    uint32_t x[16];
    tmem_ld16(sa + d, x);
    tmem_wait_ld();
    tie16(x);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(x[k]), c), m) * back);
    tmem_st16(sa + d, x);
  }
  tmem_wait_st();
}
// A warp's rows of an accumulator times each row's factor.
__device__ __noinline__ void scale_rows(uint32_t oa, int columns, float a) {
#pragma unroll 1
  for (int d = 0; d < columns; d += 16) {
    uint32_t o[16];
    tmem_ld16(oa + d, o);
    tmem_wait_ld();
    tie16(o);
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
    tmem_st16(oa + d, o);
  }
}
// The order in which a segment's tiles pass the ring: keys and values as K0 V0
// K1 V1 .. when both streams read every tile, K0 K1 V0 K2 V1 .. when they take
// turns (a stream's scores are then two tiles ahead).  Step i of 2 n.
struct Turn {
  bool is_v;
  int j;  // tile
};
__device__ __forceinline__ Turn turn_at(bool turns, int n, int i) {
  if (!turns || n == 1) return {(i & 1) != 0, i >> 1};
  if (i == 0) return {false, 0};
  if (i == 2 * n - 1) return {true, n - 1};
  return {(i & 1) == 0, (i & 1) ? (i + 1) >> 1 : (i - 2) >> 1};
}

// The same the other way round: where tile j's keys or values come, in tiles.
__device__ __forceinline__ int ring_place(bool is_v, bool turns, int n, int j) {
  if (!turns || n == 1) return 2 * j + (is_v ? 1 : 0);
  return is_v ? min(2 * j + 2, 2 * n - 1) : max(2 * j - 1, 0);
}

// The CTA's stretch of the line, entry by entry, by one warp: the requests'
// costs are summed by its lanes.
template <int NS>
struct Scheduler {
  int64_t x, x1, total;
  int q, h, pair, z, ctx, nn;
  uint32_t n;  // entries written
  bool ended;
  Cut cut;

  __device__ __forceinline__ void start(const Params &p, int lane) {
    int64_t begin, own = 0;
    const bool one_pass = p.n_req <= 32;  // a request a lane
    if (one_pass && !one_form(p)) {
      for (int b = 0; b < p.n_req; ++b) {
        int c, m;
        if (!lengths(p, b, c, m) && blockIdx.x == 0 && lane == 0) report(p.status, MFD_ERR_INPUT);
        const int64_t cost = p.cv.Hk * head_cost_warp<NS>(p, c, m, lane);
        if (lane == b) {
          own = cost;
          ctx = c;
          nn = m;
        }
        total = b ? total + cost : cost;
      }
    } else if (one_pass) {
      if (lane < p.n_req) {
        if (!lengths(p, lane, ctx, nn) && blockIdx.x == 0) report(p.status, MFD_ERR_INPUT);
        own = p.cv.Hk * head_cost<NS>(p, ctx, nn);
      }
      total = warp_total(own);
    } else {
      total = line_walk<NS>(p, lane, -1, blockIdx.x == 0, q, begin);
    }
    x = border(total, blockIdx.x, gridDim.x);
    x1 = border(total, blockIdx.x + 1, gridDim.x);
    h = pair = z = 0;
    n = 0;
    ended = false;
    cut = Cut{};
    if (x >= x1) return;
    if (one_pass) {
      const int64_t run = warp_running(own, lane);
      q = __ffs(__ballot_sync(0xffffffffu, own > 0 && x < run)) - 1;
      begin = __shfl_sync(0xffffffffu, run - own, q);
      ctx = __shfl_sync(0xffffffffu, ctx, q);
      nn = __shfl_sync(0xffffffffu, nn, q);
    } else {
      line_walk<NS>(p, lane, x, false, q, begin);
      lengths(p, q, ctx, nn);
    }
    const int64_t hc = head_cost_warp<NS>(p, ctx, nn, lane);
    h = (int)divide(x - begin, hc);
    int64_t rest = x - begin - h * hc;
    pair = find_item<NS>(p, ctx, nn, lane, rest);
    z = (int)rest;
  }
  // The next entry, to the ring and to the caller; false at the end.
  __device__ __forceinline__ bool next(const Params &p, Segment &s, int lane, Segment *ring, uint64_t *seg_full,
                                       uint64_t *seg_empty, volatile int *never) {
    if (ended) return false;
    const int st = n % SEG_RING;
    const bool room = wait_limit(&seg_empty[st], ((n / SEG_RING) & 1u) ^ 1u, 2 * kWaitLimitNs, never);
    if (!__all_sync(0xffffffffu, room)) {  // never again: the others' waits run out together
      if (lane == 0) report(p.status, MFD_ERR_TIMEOUT);
      ended = true;
      return false;
    }
    ++n;
    s.q = -1;
    ended = x >= x1;
    if (!ended) {
      const Item it = item_of<NS>(p, ctx, nn, pair);
      const int64_t left = x1 - x;
      const int end = left < it.cost - z ? z + (int)left : it.cost;
      s.q = q;
      s.h = h;
      s.pair = pair;
      s.ctx = ctx;
      s.nn = nn;
      s.active = it.active;
      s.tiles = it.tiles;
      s.t0 = tile_at(it, z);
      s.t1 = tile_at(it, end);
      s.head = z == 0;
      if (s.t0 < s.t1 && !(s.t0 == 0 && s.t1 == it.tiles)) {
        cut.has[s.t0 == 0 ? 1 : 0] = 1;
        if (s.t0 == 0) {
          cut.reach = cta_of(total, x - z + it.cost - 1, gridDim.x) - (int)blockIdx.x + 1;
          cut.q = q;
          cut.h = h;
          cut.pair = pair;
          cut.nn = nn;
        }
      }
      x += end - z;
      z = 0;
      if (end == it.cost && ++pair == p.n_pair) {
        pair = 0;
        if (++h == p.cv.Hk) {
          h = 0;
          if (++q < p.n_req) lengths(p, q, ctx, nn);
        }
      }
    }
    if (lane == 0) {
      if (ended) p.cuts[blockIdx.x] = cut;
      ring[st] = s;
      mbar_arrive(&seg_full[st]);
    }
    __syncwarp();
    return !ended;
  }
};

// Adds back what the helpers took out of the values' product: for every noted
// node from lo to hi - 1 that this row sees, the values that are not finite
// (all NaN where an E4M3 row reads back as NaN, else those that leave the
// type's range), columns d .. d + 15 in the accumulator's order.
template <typename T, bool E4M3>
__device__ __noinline__ void add_back(const Params &p, int q, int h, int ctx, int lo, int hi, int node,
                                      const uint32_t *mask_row, const uint32_t *bad, int d, uint32_t (&f)[16]) {
  const CacheView &cv = p.cv;
  for (int j = lo; j < hi; ++j) {
    if (!((bad[j >> 5] >> (j & 31)) & 1u)) continue;
    const bool sees = mask_row ? (__ldg(mask_row + (j >> 5)) >> (j & 31)) & 1u : j <= node;
    if (!sees) continue;
    const int pos = ctx + j;
    const int page = __ldg(cv.table + (size_t)q * cv.max_pages + (pos >> cv.ps_shift));
    if (page < 0 || page >= cv.n_pages) continue;
    const int slot = pos & ((1 << cv.ps_shift) - 1);
    const int64_t e = page * cv.page_stride + h * cv.head_stride + slot * cv.token_stride + d;
    if (E4M3) {
      const int code = cv.v_exp[(((int64_t)page * cv.Hk + h) << cv.ps_shift) + slot];
      const uint4 x = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(cv.v) + e);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint2 v = Widen<T>::widen4_wide(w[k], code);
        const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y);
        const float y[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (code == EXP_NAN || !(fabsf(y[i]) < INFINITY))
            f[4 * k + i] = __float_as_uint(code == EXP_NAN ? __int_as_float(0x7FFFFFFF) : __uint_as_float(f[4 * k + i]) + y[i]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint32_t w = static_cast<const uint16_t *>(cv.v)[e + k];
        if (nonfinite2<T>(w)) f[k] = __float_as_uint(__uint_as_float(f[k]) + unpack2<T>(w).x);
      }
    }
  }
}

// One E4M3 unit (128 positions x UC columns, columns from c0 of the head) to
// the swizzled operand, by 128 threads: a thread's chunks of 16 columns are at
// one column, 128 / (UC / 16) positions apart.  Two chunks at a time in a
// rolled loop (see the softmax).
template <typename T, int DP>
__device__ __forceinline__ void widen_unit(const Params &p, const uint8_t *src, uint8_t *dst, const uint16_t *power,
                                           int ht, int c0) {
  constexpr int UC = DP == 64 ? 64 : 128;
  constexpr int C = UC / 16, PER = 128 / C, K = BN / PER;  // 8 or 4 chunks a thread
  const int wide = min(p.cv.D, UC);
  const int ch = ht % C, tok0 = ht / C;
  const bool have = c0 + ch * 16 < p.cv.D;
  // Which half of its chunk a lane reads and writes first: neighbouring blocks'
  // lanes, and neighbouring positions', take opposite halves (other banks).
  const int sw = UC == 128 ? ((ch >> 2) ^ tok0) & 1 : 0;
  const uint8_t *at = src + tok0 * wide + (have ? ch * 16 : 0) + 8 * sw;
  const int flip = 8 - 16 * sw;
  // PER is a multiple of 8: the swizzle is the same for all of a thread's rows
  uint8_t *row = dst + (ch >> 2) * (BN * 128) + tok0 * 128;
  const int o1 = (((ch & 3) * 2 + sw) ^ (tok0 & 7)) << 4, o2 = (((ch & 3) * 2 + 1 - sw) ^ (tok0 & 7)) << 4;
  power += tok0;
#pragma unroll 1
  for (int k = 0; k < K; k += 2) {
    uint2 x[2], y[2];
    uint32_t pp[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      pp[e] = have ? power[e * PER] * 0x10001u : 0u;  // 0: no row or column, whatever the (finite) bytes are
      x[e] = *reinterpret_cast<const uint2 *>(at + e * PER * wide);
      y[e] = *reinterpret_cast<const uint2 *>(at + e * PER * wide + flip);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint2 a = Widen<T>::widen4(x[e].x, pp[e]), b = Widen<T>::widen4(x[e].y, pp[e]);
      *reinterpret_cast<uint4 *>(row + e * PER * 128 + o1) = make_uint4(a.x, a.y, b.x, b.y);
      const uint2 c = Widen<T>::widen4(y[e].x, pp[e]), d = Widen<T>::widen4(y[e].y, pp[e]);
      *reinterpret_cast<uint4 *>(row + e * PER * 128 + o2) = make_uint4(c.x, c.y, d.x, d.y);
    }
    at += 2 * PER * wide;
    row += 2 * PER * 128;
    power += 2 * PER;
  }
}

// The same thread's chunks again, for a unit in which some row's power of two
// has no number of the operand type: those rows, with the power applied exactly.
// Elements that leave the type's range become infinities, as they do when the row is
// read back; those of value rows from position `hide_from` on are taken out and
// their node noted (see above), since not every row of the queries sees them.
template <typename T, int DP>
__device__ __noinline__ void widen_unit_wide(const Params &p, int q, int h, int len, const uint8_t *src, uint8_t *dst,
                                             int base, bool is_v, int ht, int c0, int hide_from, uint32_t *bad,
                                             volatile int *any_bad) {
  constexpr int UC = DP == 64 ? 64 : 128;
  constexpr int C = UC / 16, PER = 128 / C, K = BN / PER;
  const CacheView &cv = p.cv;
  const int wide = min(cv.D, UC);
  const int ch = ht % C;
  if (c0 + ch * 16 >= cv.D) return;
  for (int k = 0; k < K; ++k) {
    const int tok = ht / C + k * PER, t = base + tok;
    if (t >= len) break;
    const int page = __ldg(cv.table + (size_t)q * cv.max_pages + (t >> cv.ps_shift));
    if (page < 0 || page >= cv.n_pages) continue;
    const int code = (is_v ? cv.v_exp : cv.k_exp)[(((int64_t)page * cv.Hk + h) << cv.ps_shift) +
                                                  (t & ((1 << cv.ps_shift) - 1))];
    bool odd = false;
    Widen<T>::power(code, odd);
    if (!odd) continue;
    const uint4 x = *reinterpret_cast<const uint4 *>(src + tok * wide + ch * 16);
    uint4 lo, hi;
    {
      const uint2 a = Widen<T>::widen4_wide(x.x, code), b = Widen<T>::widen4_wide(x.y, code),
                  c = Widen<T>::widen4_wide(x.z, code), d = Widen<T>::widen4_wide(x.w, code);
      lo = make_uint4(a.x, a.y, b.x, b.y);
      hi = make_uint4(c.x, c.y, d.x, d.y);
    }
    if (t >= hide_from && (any_nonfinite<T>(lo) || any_nonfinite<T>(hi))) {
      lo = without_nonfinite<T>(lo);
      hi = without_nonfinite<T>(hi);
      note_node(t - hide_from, bad, any_bad);
    }
    uint8_t *row = dst + (ch >> 2) * (BN * 128) + tok * 128;
    const int c2 = (ch & 3) * 2, x7 = tok & 7;
    *reinterpret_cast<uint4 *>(row + ((c2 ^ x7) << 4)) = lo;
    *reinterpret_cast<uint4 *>(row + (((c2 + 1) ^ x7) << 4)) = hi;
  }
}

template <typename T, int DP, bool E4M3>
__global__ void __launch_bounds__((Shape<DP, E4M3>::THREADS), 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const Params p) {
  using SH = Shape<DP, E4M3>;
  constexpr int NS = SH::NS, NU = SH::NU, NB = SH::NB, ST = SH::ST, RST = SH::RST, SG = SH::SG;
  constexpr bool SPLIT = SH::SPLIT;
  constexpr uint32_t RN = RST ? RST : 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem;
  uint8_t *sT = sQ + NS * SH::Q_TILE;
  uint8_t *sR = sT + ST * SH::STAGE;
  uint16_t *sC = reinterpret_cast<uint16_t *>(sR + RST * SH::RAW);  // E4M3 rows' powers
  uint32_t *bad = reinterpret_cast<uint32_t *>(sC + SH::POWERS / 2);  // nodes with values taken out
  uint64_t *full = reinterpret_cast<uint64_t *>(bad + MAX_N / 32);
  uint64_t *empty = full + ST;
  uint64_t *special = empty + ST;  // a unit the helpers go over before it is full (not E4M3)
  uint64_t *raw_full = special + (E4M3 ? 0 : ST);
  uint64_t *raw_empty = raw_full + RST;
  uint64_t *s_full = raw_empty + RST;
  uint64_t *p_full = s_full + 2;
  uint64_t *pv_done = p_full + 2;
  uint64_t *q_full = pv_done + 2;
  uint64_t *drain = q_full + 1;
  uint64_t *pow_full = drain + 1;
  uint64_t *pow_empty = pow_full + (E4M3 ? 4 : 0);
  uint64_t *seg_full = pow_empty + (E4M3 ? 4 : 0);
  uint64_t *seg_empty = seg_full + SEG_RING;
  Segment *seg_ring = reinterpret_cast<Segment *>(seg_empty + SEG_RING);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(seg_ring + SEG_RING);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *never = abort_flag + 1;
  volatile int *seg_done = never + 1;  // segments a softmax warpgroup has left [2]
  volatile int *any_bad = seg_done + 2;
  volatile int *wide_s = any_bad + 1;  // E4M3: a tile with a power that has no number (1 keys, 2 values) [4]

  float *top_s = reinterpret_cast<float *>(const_cast<int *>(wide_s) + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const CacheView &cv = p.cv;

  if (smem_u32(smem) & 1023u) {  // the swizzled tiles start on 1024-byte borders
    pdl_wait();  // the grid before may still read its notes
    if (tid == 0) {
      p.cuts[blockIdx.x] = Cut{};
      report(p.status, MFD_ERR_CUDA);
    }
    return;
  }
  Scheduler<NS> sched;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], E4M3 ? 4 : 1);
      mbar_init(&empty[i], 1);
      if (!E4M3) mbar_init(&special[i], 1);
    }
    for (int i = 0; i < RST; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], SPLIT ? 8 : 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < SEG_RING; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 3 + 4 * (SG + SH::HELPERS));
    }
    for (int i = 0; i < (E4M3 ? 4 : 0); ++i) {
      mbar_init(&pow_full[i], 1);
      mbar_init(&pow_empty[i], 8 * NU);  // four warps for each of a tile's units
    }
    mbar_init(q_full, 4 * SG);
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
  tc_fence_before();
  block_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Not before the CTA has its tensor memory: a grid launched from here on may ask
  // for some on the same SM and keep it until this grid has ended.
  pdl_launch_dependents();
  pdl_wait();  // the setup above may overlap the previous grid; all that follows reads global memory

  Segment s;
  uint32_t seg_n = 0;
  bool ok = true;
  // A wait that ran out, or was told to stop, ends the CTA's work: every role
  // goes on through its list without waiting or touching anything.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (ok && !try_wait_sleep(bar, parity)) ok = wait_or_abort(bar, parity, abort_flag, p.status);
  };
  // The next entry; `arrive`: the thread that says it has been read.
  auto next_segment = [&](bool arrive) {
    const int st = seg_n % SEG_RING;
    if (!wait_limit(&seg_full[st], (seg_n / SEG_RING) & 1u, SEG_LIMIT_NS, never)) return false;
    s = seg_ring[st];
    ++seg_n;
    if (!arrive) return s.q >= 0;
    mbar_arrive(&seg_empty[st]);
    return s.q >= 0;
  };
  // The same for a warp.
  auto next_segment_warp = [&]() {
    const int st = seg_n % SEG_RING;
    const bool got = wait_limit(&seg_full[st], (seg_n / SEG_RING) & 1u, SEG_LIMIT_NS, never);
    if (!__all_sync(0xffffffffu, got)) return false;
    s = seg_ring[st];
    ++seg_n;
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[st]);
    return s.q >= 0;
  };
  // The noted nodes serve a segment until its rows are out: waits until the
  // softmax warpgroups have left `seg` segments.
  auto wait_rows_out = [&](int seg) {
    if (!ok) return;
    const unsigned long long t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
      if (seg_done[0] >= seg && (SG == 1 || seg_done[1] >= seg)) return;
      if ((it & 15u) == 0 && (*abort_flag || globaltimer() - t0 > kWaitLimitNs)) {
        if (!*abort_flag) report(p.status, MFD_ERR_TIMEOUT);
        *abort_flag = 1;
        ok = false;
        return;
      }
      __nanosleep(64);
    }
  };
  if (warp < 4) {
    if (warp == 0 || warp == 3) {
      // ------------------------------------------------------- loads
      // Warp 0 the keys, warp 3 the values: one warp for both took about 1.6 us
      // over a unit of small pages (looking them up, waits, copies), longer than
      // the rest of the SM over the tile.
      const bool is_v = warp == 3;
      const CUtensorMap *map = is_v ? &map_v : &map_k;
      // Keys and values of one token serve M rows of this CTA only, or of
      // neighbours too when there are more row tiles: then they stay in L2.
      const uint64_t policy = p.n_pair > 1 ? policy_evict_normal() : policy_evict_first();
      const int row_shift = min(cv.ps_shift, 7), rows = 1 << row_shift;  // of a box
      const uint32_t wide = E4M3 ? (uint32_t)min(cv.D, SH::UC) : 128u;   // bytes of a row in the unit
      constexpr uint32_t RING = E4M3 ? RN : ST, UNIT = E4M3 ? SH::RAW : SH::STAGE;
      // The ring's places are both warps' in the units' order (16-bit caches: the
      // ring that the MMAs read), or half of them each warp's own (8-bit ones).
      const uint32_t st0 = E4M3 && is_v ? RN / 2 : 0, st1 = E4M3 ? st0 + RN / 2 : ST;
      const uint32_t ring = smem_u32(E4M3 ? sR : sT), ready = smem_u32(E4M3 ? raw_full : full);
      uint64_t *freed = E4M3 ? raw_empty : empty;
      uint32_t st = st0, par = 0;  // ring place and its phase
      uint32_t special_par = 0, issued = 0, issued_special = 0, issued_par = 0;
      auto next_place = [&]() {
        if (++st == st1) {
          st = st0;
          par ^= 1u;
        }
      };
      // Past the other warp's units in the shared ring.  A wait for a place must
      // not come a phase early or late, when a parity passes for another phase's:
      // the MMAs free places in order, and no two units of a warp are further apart
      // than the ring is long, so its last wait vouches for the phase before last.
      // The two groups of helpers free places in no common order, so in the 8-bit
      // rings every place's every phase is waited for by the warp that fills it.
      auto skip = [&](int units) {
        for (; !E4M3 && units > 0; --units) next_place();
      };
      while (next_segment_warp()) {
        const int nt = s.t1 - s.t0;
        const bool turns = s.active != 2;
        const int len = s.ctx + s.nn;
        const int32_t *table = cv.table + (size_t)s.q * cv.max_pages;
        // a lane's box of tile j; its page is looked up a tile ahead
        auto page_at = [&](int j) {
          const int t = (s.t0 + j) * BN + (lane << row_shift);
          int page = 0;
          if (j < nt && (lane << row_shift) < BN && t < len) {
            page = __ldg(table + (t >> cv.ps_shift));
            if ((unsigned)page >= (unsigned)cv.n_pages) {
              report(p.status, MFD_ERR_INPUT);
              page = cv.n_pages;  // outside the map: reads as zeros
            }
          }
          return page;
        };
        int page_next = page_at(0);
        int at = 0;  // tiles of the segment that have passed
        for (int j = 0; j < nt; ++j) {
          const int place = ring_place(is_v, turns, nt, j);
          skip((place - at) * NU);
          at = place + 1;
          const int base = (s.t0 + j) * BN;
          const int page = page_next;
          page_next = page_at(j + 1);
          const int some = (min(len - base, BN) + rows - 1) >> row_shift;  // boxes with positions before the end
          const int slot = base & ((1 << cv.ps_shift) - 1);  // of the first box; boxes of smaller pages start at 0
          const bool sp = !E4M3 && is_v && base + BN > s.ctx;
#pragma unroll 1
          for (int u = 0; u < NU; ++u) {
            wait(&freed[st], par ^ 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              const uint32_t bar = sp ? smem_u32(&special[st]) : ready + st * 8;
              uint32_t dst = ring + st * UNIT;
              const bool one = elect_one();
              if (one) expect_bytes(bar, (uint32_t)some * rows * wide * (E4M3 ? 1 : NB));
              for (int b = 0; b < some; ++b, dst += rows * wide) {
                const int pg = __shfl_sync(0xffffffffu, page, b);
                if (one) {
                  tma_load_4d(dst, map, u * SH::UC, slot, s.h, pg, bar, policy);
                  if (!E4M3 && NB == 2) tma_load_4d(dst + BN * 128, map, u * SH::UC + 64, slot, s.h, pg, bar, policy);
                }
              }
              const uint32_t bit = 1u << st;
              issued |= bit;
              issued_par = (sp ? (special_par & bit) != 0 : par != 0) ? issued_par | bit : issued_par & ~bit;
              issued_special = sp ? issued_special | bit : issued_special & ~bit;
              if (sp) special_par ^= bit;
            }
            next_place();
          }
        }
        skip((2 * nt - at) * NU);
      }
      // Every load issued lands before the CTA may exit.  All have been consumed
      // unless a wait ran out; a place that the other warp has filled since holds
      // this warp's load no more, and its wait then runs out too.
      if (!ok && lane == 0)
        for (uint32_t i = 0; i < RING; ++i)
          if ((issued >> i) & 1u)
            mbar_wait(E4M3 ? &raw_full[i] : ((issued_special >> i) & 1u) ? &special[i] : &full[i],
                      (issued_par >> i) & 1u, never);
      __syncwarp();
    } else if (warp == 1) {
      if (elect_one()) {
        // ----------------------------------------------------- MMAs
        constexpr uint32_t id_s = idesc_16<T>(BM, BN, false), id_o = idesc_16<T>(BM, SH::UC, true);
        uint32_t st = 0, par = 0;  // ring place and its phase
        uint32_t q_par = 0, p_par = 0;
        while (next_segment(true)) {
          const int nt = s.t1 - s.t0;
          if (nt == 0) continue;
          const bool shared = s.active == 2;
          const int steps = shared ? 2 * nt : nt;
          wait(q_full, q_par);
          q_par ^= 1u;
          uint32_t kst = 0, vst = 0;
          auto take = [&]() {
            const uint32_t now = st;
            wait(&full[st], par);
            if (++st == ST) {
              st = 0;
              par ^= 1u;
            }
            return now;
          };
          auto scores = [&](int i) {
            const uint32_t d = tmem + SH::TM_S + (uint32_t)(i & 1) * BN;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
              if (!shared || !(i & 1)) kst = take();
              if (!ok) continue;
              tc_fence_after();
              const uint32_t qa =
                  desc_lo(smem_u32(sQ) + (shared ? (uint32_t)(i & 1) * SH::Q_TILE : 0u) + u * (NB * BM * 128), 16);
              const uint32_t ka = desc_lo(smem_u32(sT) + kst * SH::STAGE, 16);
              const int k_steps = min(cv.D - u * SH::UC, SH::UC) / 16;
#pragma unroll
              for (int k = 0; k < SH::UC / 16; ++k)
                if (k < k_steps)
                  mma_ss(d, qa + (k >> 2) * (BM * 128 >> 4) + (k & 3) * 2, ka + (k >> 2) * (BN * 128 >> 4) + (k & 3) * 2,
                         id_s, u != 0 || k != 0);
              if (!shared || (i & 1)) tc_commit(&empty[kst]);
            }
            if (ok) tc_commit(&s_full[i & 1]);
          };
          auto values = [&](int i) {
            wait(&p_full[i & 1], (p_par >> (i & 1)) & 1u);
            p_par ^= 1u << (i & 1);
            const int acc = NS == 2 ? i & 1 : 0;
            const uint32_t a = tmem + SH::TM_S + (uint32_t)(i & 1) * BN;
            const bool more = NS == 2 ? i >= 2 : i >= 1;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
              if (!shared || !(i & 1)) vst = take();
              if (!ok) continue;
              tc_fence_after();
              const uint32_t va = desc_lo(smem_u32(sT) + vst * SH::STAGE, BN * 128);
              const uint32_t d = tmem + SH::TM_O + (uint32_t)(acc * DP + u * SH::UC);
#pragma unroll
              for (int k = 0; k < BN / 16; ++k) mma_ts(d, a + k * 8 + (SPLIT && k >= 4 ? 32 : 0), va + k * (2048 >> 4), id_o, more || k != 0);
              if (!shared || (i & 1)) tc_commit(&empty[vst]);
            }
            if (ok) tc_commit(&pv_done[acc]);
          };
          // one place each in the code for scores and values
          for (int i = -2; i < steps; ++i) {
            if (i >= 0) values(i);
            if (i + 2 < steps) scores(i + 2);
          }
        }
        tc_commit(drain);  // all MMAs finish before tensor memory is released
        mbar_wait(drain, 0, never);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------- list of work
      // E4M3: also the exponent bytes of every tile's positions, four a lane, as powers
      // for the helpers.
      if (lane == 0) p.cuts[blockIdx.x] = Cut{};  // stands if a wait runs out before the list's end
      sched.start(p, lane);
      uint32_t n = 0;
      int seg = 0;
      while (sched.next(p, s, lane, seg_ring, seg_full, seg_empty, never)) {
        const int nt = s.t1 - s.t0;
        if (!E4M3 || nt == 0) continue;
        const int len = s.ctx + s.nn;
        const bool note = p.N > 1 || p.mask;
        bool clean = false;
        const int32_t *table = cv.table + (size_t)s.q * cv.max_pages;
        auto page_at = [&](int t) { return t < min(len, s.t1 * BN) ? __ldg(table + (t >> cv.ps_shift)) : -1; };
        int page[4], ck[4], cw[4];  // pages two tiles ahead, bytes one tile ahead
        auto load = [&](int t0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = t0 + 32 * i + lane;
            ck[i] = cw[i] = -1;
            if (page[i] >= 0 && page[i] < cv.n_pages) {
              const int64_t e = (((int64_t)page[i] * cv.Hk + s.h) << cv.ps_shift) + (t & ((1 << cv.ps_shift) - 1));
              ck[i] = __ldg(cv.k_exp + e);
              cw[i] = __ldg(cv.v_exp + e);
            }
            page[i] = page_at(t + BN);
          }
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) page[i] = page_at(s.t0 * BN + 32 * i + lane);
        load(s.t0 * BN);
        for (int j = 0; j < nt; ++j, ++n) {
          const int base = (s.t0 + j) * BN, slot = n & 3;
          int now_k[4], now_v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            now_k[i] = ck[i];
            now_v[i] = cw[i];
          }
          load(base + BN);
          if (note && base + BN > s.ctx && !clean) {
            wait_rows_out(seg);
            for (int k = lane; k < MAX_N / 32; k += 32) bad[k] = 0;
            if (lane == 0) *any_bad = 0;
            __syncwarp();
            clean = true;
          }
          wait(&pow_empty[slot], ((n >> 2) & 1u) ^ 1u);
          ok = __all_sync(0xffffffffu, ok);
          bool wk = false, wv = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = base + 32 * i + lane;
            const uint16_t pk = now_k[i] < 0 ? 0 : Widen<T>::power(now_k[i], wk);
            uint16_t pv = now_v[i] < 0 ? 0 : Widen<T>::power(now_v[i], wv);
            if (now_v[i] == EXP_NAN && note && t >= s.ctx) {
              // a NaN that some rows do not see: out of the product, added back later
              pv = 0;
              note_node(t - s.ctx, bad, any_bad);
            }
            if (ok) {
              sC[slot * BN + 32 * i + lane] = pk;
              sC[4 * BN + slot * BN + 32 * i + lane] = pv;
            }
          }
          const int w = (__any_sync(0xffffffffu, wk) ? 1 : 0) | (__any_sync(0xffffffffu, wv) ? 2 : 0);
          if (lane == 0 && ok) {
            wide_s[slot] = w;
            mbar_arrive(&pow_full[slot]);
          }
          __syncwarp();
        }
        ++seg;
      }
    }
  } else if (warp < SH::HELP_WARP) {
    // --------------------------------------------------------- softmax
    const int ws = SG == 2 ? (warp - 4) >> 2 : 0;  // stream, or half of a stream's columns (SPLIT)
    const int wq = warp & 3;                       // the warp's lanes of tensor memory
    const int r = wq * 32 + lane;
    const int acc = NS == 2 ? ws : 0;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    constexpr int S_COLS = SPLIT ? BN / 2 : BN, O_COLS = SPLIT ? DP / 2 : DP;  // this thread's
    const int s_col = SPLIT ? ws * S_COLS : 0;
    const uint32_t o_base = lane_base + SH::TM_O + (uint32_t)ws * O_COLS;
    uint32_t s_par = 0, pv_n = 0;
    // alternating streams exchange (m, l) in the space of the second Q tile
    float2 *ml_s = reinterpret_cast<float2 *>(sQ + (NS - 1) * SH::Q_TILE);
    while (next_segment_warp()) {
      const int nt = s.t1 - s.t0;
      const bool shared = s.active == 2;
      const int live = s.nn * p.G;
      const int rt = shared ? ws : 0;                     // row tile of the group
      const int row0 = (s.pair * NS + rt) * BM;
      const int row = row0 + r;                           // this thread's row
      const int node = row / p.G, g = row - node * p.G;
      const bool row_live = row < live && nt > 0;
      const bool warp_live = row0 + wq * 32 < live && nt > 0;

      // queries: 16-byte chunks to the swizzled tile; rows that are not live
      // stay as they are (a row's scores reach no other row)
      if (nt > 0) {
        constexpr int C = DP / 8, STEP = 128 / C;
        const bool all = shared || SG == 1;  // else half the rows each
        const int base_row = all ? 0 : ws * (BM / 2);
        const int have = min(all ? BM : BM / 2, live - row0 - base_row);  // rows to load
        const int ch = r % C;
        const uint32_t dst = smem_u32(sQ + rt * SH::Q_TILE) + (ch >> 3) * (BM * 128);
        const uint16_t *src = p.q + (int64_t)s.q * p.N * p.q_stride + (int64_t)s.h * p.G * cv.D + ch * 8;
        if (ch * 8 < cv.D && r / C < have) {
          int i = r / C;
          int n1 = (row0 + base_row + i) / p.G, g1 = row0 + base_row + i - n1 * p.G;
          const int dn = STEP / p.G, dg = STEP - dn * p.G;
#pragma unroll 1
          for (; i < have; i += 4 * STEP) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int rr = base_row + i + b * STEP;
              const uint16_t *at = src + n1 * p.q_stride + g1 * cv.D;
              if (i + b * STEP < have) cp_async16(dst + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4), at);
              n1 += dn;
              g1 += dg;
              if (g1 >= p.G) {
                g1 -= p.G;
                ++n1;
              }
            }
          }
          if (E4M3) {  // into the widened keys' order: a thread's own chunks, once they are here
            cp_async_wait();
#pragma unroll 4
            for (int rr = base_row + r / C; rr < base_row + have; rr += STEP) {
              const uint32_t at = dst + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
              const uint4 x = ld_shared16(at);
              st_shared16(at, make_uint4(__byte_perm(x.x, x.y, 0x7632), __byte_perm(x.x, x.y, 0x5410),
                                         __byte_perm(x.z, x.w, 0x7632), __byte_perm(x.z, x.w, 0x5410)));
            }
          }
        }
      }
      // rows past n_nodes, once per item: zeros and -infinity
      if (s.head && (NS == 2 || ws == 0)) {
        const int first = (s.pair * NS + acc) * BM + wq * 32, c8 = cv.D / 8;
        const int lo = max(first, s.tiles ? live : 0), rows = min(first + 32, p.M) - lo;
#pragma unroll 1
        for (int i = lane; i < rows * c8; i += 32) {
          const int rr = lo + i / c8, ch = i % c8;
          const int zn = rr / p.G, zg = rr - zn * p.G;
          const int64_t at = ((int64_t)s.q * p.N + zn) * p.Hq + s.h * p.G + zg;
          st_global16(p.out + at * cv.D + ch * 8, make_uint4(0, 0, 0, 0));
          if (ch == 0 && p.lse) p.lse[at] = -INFINITY;
        }
      }
      if (nt == 0) continue;
      cp_async_wait();
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
        uint32_t vis[S_COLS / 32];
        bool hide = false;
        if (t_base + BN > s.ctx && warp_live) {
          uint32_t every = 0xFFFFFFFFu;
#pragma unroll
          for (int k = 0; k < S_COLS / 32; ++k) {
            vis[k] = row_live ? visible32(mask_row, p.W32, node, s.nn, t_base + s_col + 32 * k - s.ctx) : 0xFFFFFFFFu;
            every &= vis[k];
          }
          hide = __any_sync(0xffffffffu, every != 0xFFFFFFFFu);
        }
        wait(&s_full[slot], (s_par >> slot) & 1u);
        s_par ^= 1u << slot;
        ok = __all_sync(0xffffffffu, ok);
        const uint32_t sa = lane_base + SH::TM_S + (uint32_t)(slot * BN + s_col);
        constexpr int SW = SH::SW;
        float top = -INFINITY;
        if (ok && warp_live) {
          tc_fence_after();
          if (hide) hide_scores(sa, S_COLS, vis[0], vis[1], vis[S_COLS / 32 - 2], vis[S_COLS / 32 - 1]);
          // Both passes read the scores from tensor memory, 32 columns at a time
          // in a rolled loop: 128 in registers took unrolled code for all of
          // them, and the warps then waited for instructions (3.5 cycles an
          // issue) more than for anything else.
#pragma unroll 1
          for (int part = 0; part < S_COLS / SW; ++part) {
            uint32_t x[SW];
#pragma unroll
            for (int k = 0; k < SW; k += 32) tmem_ld32(sa + SW * part + k, x + k);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < SW; k += 32) tie32(x + k);
            float t[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < SW; k += 2)
              t[(k >> 1) & 3] = max3(t[(k >> 1) & 3], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
            top = max3(max3(t[0], t[1], t[2]), t[3], top);
          }
        }
        if (SPLIT) {  // the row's maximum over both halves
          float *mine = top_s + (i & 1) * (2 * BM) + r;
          mine[ws * BM] = top;
          named_sync(1, 256);
          top = fmaxf(top, mine[(ws ^ 1) * BM]);
        }
        if (ok && warp_live) {
          top *= p.c;
          // move the maximum when it has grown by enough (or is the first)
          const bool move = row_live && top > m + MAX_GROWTH;
          if (__any_sync(0xffffffffu, move)) {
            const float m2 = move ? top : m;
            const float a = move ? ex2(m - m2) : 1.f;
            m = m2;
            l *= a;
            if (done) {
              wait(&pv_done[acc], (pv_n - 1u) & 1u);
              tc_fence_after();
              scale_rows(o_base, O_COLS, a);
            }
          }
          float mz = m == -INFINITY ? 0.f : m;
          if (__any_sync(0xffffffffu, fabsf(mz) > LARGE_SCORE)) {
            center_scores(sa, S_COLS, p.c, mz);
            mz = 0.f;
          }
          const uint64_t cc = pair(p.c, p.c), mm = pair(-mz, -mz);
          uint64_t sum0 = pair(0.f, 0.f), sum1 = sum0;
#pragma unroll 1
          for (int part = 0; part < S_COLS / SW; ++part) {
            uint32_t x[SW];
#pragma unroll
            for (int k = 0; k < SW; k += 32) tmem_ld32(sa + SW * part + k, x + k);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < SW; k += 32) tie32(x + k);
#pragma unroll
            for (int c = 0; c < SW; c += 32) {
              uint32_t pk[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 y =
                    unpair(fma2(pair(__uint_as_float(x[c + 2 * k]), __uint_as_float(x[c + 2 * k + 1])), cc, mm));
                const float a = ex2(y.x), b = ex2(y.y);
                if (k & 1)
                  sum1 = add2(sum1, pair(a, b));
                else
                  sum0 = add2(sum0, pair(a, b));
                pk[k] = pack2<T>(a, b);  // the type that the product takes; the sum has them unrounded
              }
              tmem_st16(sa + (SW * part + c) / 2, pk);  // over scores that have been read
            }
          }
          const float2 sum = unpair(add2(sum0, sum1));
          l += sum.x + sum.y;
          tmem_wait_st();
        }
        // With one stream scores are two tiles ahead of the products, and the last
        // but one may still run.  It is waited for before the last can start: a
        // wait on a parity is for the one phase that is open.
        if (NS == 1 && done && i + 1 == steps) wait(&pv_done[acc], (pv_n - 1u) & 1u);
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&p_full[slot]);
        ++done;
        ++pv_n;
      }

      // ------------------------------------------------------- epilogue
      if (done) wait(&pv_done[acc], (pv_n - 1u) & 1u);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const bool alternating = NS == 2 && !shared;
      float a0 = 1.f, a1 = 0.f;
      if (alternating) {
        ml_s[ws * BM + r] = make_float2(m, l);
        named_sync(1, 256);
        const float2 f = ml_s[r], o = ml_s[BM + r];
        m = fmaxf(f.x, o.x);
        if (m > -INFINITY) {
          a0 = f.x == -INFINITY ? 0.f : ex2(f.x - m);
          a1 = o.x == -INFINITY ? 0.f : ex2(o.x - m);
          l = f.y * a0 + o.y * a1;
        } else {
          l = f.y + o.y;  // nothing seen (0), or NaN
        }
      }
      if (SPLIT) {
        float *mine = top_s + (steps & 1) * (2 * BM) + r;
        mine[ws * BM] = l;
        named_sync(1, 256);
        l = mine[0] + mine[BM];
      }
      const bool whole = s.t0 == 0 && s.t1 == s.tiles;
      if (ok && warp_live) {
        const bool two = alternating && steps > 1;
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          a0 *= inv;
          a1 *= inv;
        }
        // columns: all of this stream's, or half of the two streams' sum, or
        // this warpgroup's half of the one stream's
        const bool half = alternating || SPLIT;
        const int middle = SPLIT ? O_COLS : (cv.D + 31) / 32 * 16;
        const int d0 = half && ws == 1 ? middle : 0, d1 = half && ws == 0 ? min(middle, cv.D) : cv.D;
        const uint32_t from = alternating ? lane_base + SH::TM_O : o_base - (SPLIT ? ws * O_COLS : 0);
        const int64_t at = row_live ? ((int64_t)s.q * p.N + node) * p.Hq + s.h * p.G + g : 0;
        const int part = 2 * (int)blockIdx.x + (s.t0 == 0 ? 1 : 0);
        const bool fix = (p.N > 1 || p.mask) && s.t1 * BN > s.ctx && *any_bad;
        float4 *po = p.part_o + (int64_t)part * (cv.D / 4) * p.part_rows + rt * BM + r;
        // a row's place: 16 columns are 32 bytes of the output, or 4 of its
        // part's float4, each the rows' length from the next
        const int64_t hop = (int64_t)p.part_rows * 16;
        uint8_t *dst = whole ? reinterpret_cast<uint8_t *>(p.out + at * cv.D + d0) : reinterpret_cast<uint8_t *>(po) + hop * (d0 / 4);
#pragma unroll 1
        for (int d = d0; d < d1; d += 16) {
          uint32_t o[16];
          tmem_ld16(from + d, o);
          if (two) {
            uint32_t o1[16];
            tmem_ld16(from + DP + d, o1);
            tmem_wait_ld();
            tie16(o);
            tie16(o1);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              o[k] = __float_as_uint(fmaf(__uint_as_float(o1[k]), a1, __uint_as_float(o[k]) * a0));
          } else {
            tmem_wait_ld();
            tie16(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a0);
          }
          if (fix && row_live)
            add_back<T, E4M3>(p, s.q, s.h, s.ctx, max(0, s.t0 * BN - s.ctx), min(s.nn, s.t1 * BN - s.ctx), node, mask_row,
                              bad, d, o);
          // E4M3: columns 4 i .. 4 i + 3 were widened in the order 1, 3, 0, 2
          auto f = [&](int k) {
            constexpr int FROM[4] = {E4M3 ? 2 : 0, E4M3 ? 0 : 1, E4M3 ? 3 : 2, E4M3 ? 1 : 3};
            return __uint_as_float(o[(k & ~3) + FROM[k & 3]]);
          };
          if (row_live) {
            if (whole) {
              st_global16(dst, make_uint4(pack2<T>(f(0), f(1)), pack2<T>(f(2), f(3)), pack2<T>(f(4), f(5)), pack2<T>(f(6), f(7))));
              st_global16(dst + 16,
                          make_uint4(pack2<T>(f(8), f(9)), pack2<T>(f(10), f(11)), pack2<T>(f(12), f(13)), pack2<T>(f(14), f(15))));
              dst += 32;
            } else {
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                st_global16(dst, make_uint4(__float_as_uint(f(k)), __float_as_uint(f(k + 1)), __float_as_uint(f(k + 2)),
                                            __float_as_uint(f(k + 3))));
                dst += hop;
              }
            }
          }
        }
        if (row_live && !(half && ws == 1)) {
          if (!whole)
            p.part_ml[(int64_t)part * p.part_rows + rt * BM + r] = make_float2(m, l);
          else if (p.lse)
            p.lse[at] = l == 0.f ? -INFINITY : m * LN2 + logf(l);
        }
      }
      tc_fence_before();
      if (alternating) named_sync(1, 256);  // each has read the other's O and (m, l)
      tc_fence_after();
      if (p.N > 1 || p.mask) {  // the noted nodes are read: the helpers may clear them
        if (ws == 0)
          named_sync(2, 128);
        else
          named_sync(3, 128);
        if (r == 0) {
          __threadfence_block();
          seg_done[ws] = seg_done[ws] + 1;
        }
      }
    }
  } else {
    // --------------------------------------------------------- helpers
    // E4M3: the two warpgroups take the units in turn
    const int ht = (tid - SH::HELP_WARP * 32) & 127, hg = (tid - SH::HELP_WARP * 32) >> 7;
    uint32_t unit = 0;
    uint32_t st = 0, par = 0;  // place in the MMAs' ring and its phase
    // The same in the loaders' rings of keys and of values.  A group waits only for
    // its own units there; by then the MMAs have read the unit a ring of theirs
    // before, so the place's previous unit was loaded (with two units a tile, it
    // was the group's own).
    uint32_t rk = 0, rk_par = 0, rv = RN / 2, rv_par = 0;
    uint32_t special_par = 0, pow_n = 0;
    int seg = 0;
    while (next_segment_warp()) {
      const int nt = s.t1 - s.t0;
      if (nt == 0) continue;
      const bool turns = s.active != 2;
      const int len = s.ctx + s.nn;
      // one row without a mask sees every key before the end
      const bool note = p.N > 1 || p.mask;
      bool clean = false;  // the bad-node bits are this segment's
      // bf16 and fp16: only value tiles that reach past the context
      for (int i = 0; i < 2 * nt; ++i) {
        const Turn tn = turn_at(turns, nt, i);
        const bool is_v = tn.is_v;
        const int j = tn.j;
        const int base = (s.t0 + j) * BN;
        const bool sp = is_v && base + BN > s.ctx;
        if (!E4M3 && sp && note && !clean) {
          wait_rows_out(seg);
          named_sync(4, 128);
          for (int k = ht; k < MAX_N / 32; k += 128) bad[k] = 0;
          if (ht == 0) *any_bad = 0;
          named_sync(4, 128);
          clean = true;
        }
        const uint32_t pn = pow_n + j;
#pragma unroll 1
        for (int u = 0; u < NU; ++u) {
          const uint32_t rs = is_v ? rv : rk, rpar = is_v ? rv_par : rk_par;
          if (E4M3 && is_v && ++rv == RN) {
            rv = RN / 2;
            rv_par ^= 1u;
          }
          if (E4M3 && !is_v && ++rk == RN / 2) {
            rk = 0;
            rk_par ^= 1u;
          }
          if (E4M3 && (int)(unit++ & 1u) != hg) {
            // the other group's
          } else if (E4M3) {
            wait(&pow_full[pn & 3], (pn >> 2) & 1u);
            wait(&empty[st], par ^ 1u);
            wait(&raw_full[rs], rpar);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              widen_unit<T, DP>(p, sR + rs * SH::RAW, sT + st * SH::STAGE, sC + (is_v ? 4 * BN : 0) + (pn & 3) * BN, ht,
                                u * SH::UC);
              if ((wide_s[pn & 3] >> (is_v ? 1 : 0)) & 1)
                widen_unit_wide<T, DP>(p, s.q, s.h, len, sR + rs * SH::RAW, sT + st * SH::STAGE, base, is_v, ht, u * SH::UC,
                                       is_v && note ? s.ctx : INT_MAX, bad, any_bad);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && ok) {
              mbar_arrive(&raw_empty[rs]);
              mbar_arrive(&full[st]);
              mbar_arrive(&pow_empty[pn & 3]);
            }
          } else if (sp) {
            wait(&special[st], (special_par >> st) & 1u);
            special_par ^= 1u << st;
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              uint8_t *dst = sT + st * SH::STAGE;
              constexpr int C = SH::UC / 8, PER = 128 / C;
              const int ch = ht % C;
#pragma unroll 4
              for (int tok = ht / C; tok < BN; tok += PER) {
                const int t = base + tok;
                uint4 *at = reinterpret_cast<uint4 *>(dst + (ch >> 3) * (BN * 128) + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
                if (t >= len) {
                  *at = make_uint4(0, 0, 0, 0);
                } else if (note && t >= s.ctx) {
                  const uint4 x = *at;
                  if (any_nonfinite<T>(x)) {
                    *at = without_nonfinite<T>(x);
                    note_node(t - s.ctx, bad, any_bad);
                  }
                }
              }
            }
            fence_async_smem();
            named_sync(4, 128);
            if (ht == 0 && ok) mbar_arrive(&full[st]);
          }
          if (++st == ST) {
            st = 0;
            par ^= 1u;
          }
        }
      }
      ++seg;
      pow_n += nt;
    }
  }
  tc_fence_before();
  block_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join

constexpr int JOIN_ROWS = 16;

// Combines the parts of the items that borders cut.  Block (c, y): the item
// whose first part CTA c holds, if any, and 16 of its rows: first the notes of
// the CTAs that may hold parts, then every part's (m, l), from which its weight
// 2^(m - max m) / sum comes, then the parts' O.  A thread adds up one row's 8
// columns, and where the block has few rows (one token) several threads share
// the parts; the order is the parts', whatever CTA was done first.  It waits for
// its loads, one round after the other: it is 5 us of the 15 of one token over
// 700 positions (nine parts for each of 8 heads), 7 of the 129 over 200,002
// (19 each), 10 of one tree's 61, whose parts are 20 MB.
template <typename T, int NS>
__global__ void __launch_bounds__(JOIN_ROWS * 32) join_kernel(const Params p) {
  __shared__ float w_s[ATTENTION_MAX_CTAS][JOIN_ROWS];
  __shared__ int slot_s[ATTENTION_MAX_CTAS];
  __shared__ float4 sum_s[2][JOIN_ROWS * 32];
  const int tid = threadIdx.x, lane = tid & 31, chunks = p.cv.D / 8, threads = JOIN_ROWS * chunks;
  pdl_launch_dependents();
  pdl_wait();  // the parts are written
  const int c0 = blockIdx.x;
  const Cut cut = p.cuts[c0];
  const bool usable = cut_usable(cut, c0, (int)gridDim.x, p.n_req, p.cv.Hk, p.n_pair, p.N);
  const int n_part = cut.reach, q = cut.q, h = cut.h;
  // each part's slot, or -1 where a CTA's stretch of the item holds no key tile
  auto note = [&](int i) { slot_s[i] = i == 0 ? 2 * c0 + 1 : p.cuts[c0 + i].has[0] ? 2 * (c0 + i) : -1; };
  if (tid < 8 && c0 + tid < (int)gridDim.x) note(tid);  // before it is known how many there are
  const int first = cut.pair * NS * BM;
  const int row0 = (int)blockIdx.y * JOIN_ROWS;
  const int rows = min(min(cut.nn * p.G - first, NS * BM) - row0, JOIN_ROWS);  // of this block
  if (!usable || rows <= 0) return;
  for (int i = 8 + tid; i < n_part; i += threads) note(i);
  block_sync();
  // a thread's row, columns, and every `groups`th part from its own
  const int per = rows > 8 ? 16 : rows > 4 ? 8 : rows > 2 ? 4 : rows;  // 1, 2, 4, 8 or 16
  const int groups = JOIN_ROWS / per;
  const int r = tid % per, ch = tid / per % chunks, group = tid / per / chunks;
  const bool have = r < rows;
  // weights: G threads for each row
  const int G = p.cv.D >= 128 ? 16 : p.cv.D >= 64 ? 8 : p.cv.D >= 32 ? 4 : 2;
  if (tid < JOIN_ROWS * G) {
    const int r = tid / G, j = tid % G, row = row0 + r;
    const unsigned peers = ((1u << G) - 1u) << (lane / G * G);
    float m = -INFINITY;
    for (int i = j; i < n_part; i += G)
      if (slot_s[i] >= 0 && r < rows) m = fmaxf(m, p.part_ml[(int64_t)slot_s[i] * p.part_rows + row].x);
    for (int o = G / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(peers, m, o));
    float l = 0.f;
    for (int i = j; i < n_part; i += G) {
      float w = 0.f;
      if (slot_s[i] >= 0 && r < rows) {
        const float2 ml = p.part_ml[(int64_t)slot_s[i] * p.part_rows + row];
        // a part whose keys are not seen has sum 0; one whose scores are NaN a NaN
        w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : ml.y) : ex2(ml.x - m);
        l += w * ml.y;
        if (w == 0.f && ml.x > -INFINITY) w = TINY_WEIGHT;
      }
      w_s[i][r] = w;
    }
    for (int o = G / 2; o > 0; o >>= 1) l += __shfl_xor_sync(peers, l, o);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = j; i < n_part; i += G) w_s[i][r] = join_weight(slot_s[i], w_s[i][r], inv);
    if (r < rows && p.lse && j == 0) {
      const int node = (first + row) / p.G, g = first + row - node * p.G;
      p.lse[((int64_t)q * p.N + node) * p.Hq + h * p.G + g] = l == 0.f ? -INFINITY : m * LN2 + logf(l);
    }
  }
  block_sync();
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll 4
  for (int i = group; i < n_part; i += groups) {
    const float w = have ? w_s[i][r] : 0.f;  // 0 where there is no part, or the row sees nothing of it
    if (w == 0.f) continue;
    const float4 *o = p.part_o + ((int64_t)slot_s[i] * (p.cv.D / 4) + 2 * ch) * p.part_rows + row0 + r;
    float4 a = o[0], b = o[p.part_rows];
    if (w == TINY_WEIGHT) {  // only what is not finite counts; an infinity's sign is the weight's, times -1 below
      auto only = [](float x) { return fabsf(x) < INFINITY ? 0.f : -x; };
      a = make_float4(only(a.x), only(a.y), only(a.z), only(a.w));
      b = make_float4(only(b.x), only(b.y), only(b.z), only(b.w));
    }
    acc[0] = fmaf(w, a.x, acc[0]);
    acc[1] = fmaf(w, a.y, acc[1]);
    acc[2] = fmaf(w, a.z, acc[2]);
    acc[3] = fmaf(w, a.w, acc[3]);
    acc[4] = fmaf(w, b.x, acc[4]);
    acc[5] = fmaf(w, b.y, acc[5]);
    acc[6] = fmaf(w, b.z, acc[6]);
    acc[7] = fmaf(w, b.w, acc[7]);
  }
  if (groups > 1) {
    sum_s[0][tid] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    sum_s[1][tid] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    block_sync();
    if (group > 0) return;
    for (int k = 1; k < groups; ++k) {
      const float4 x = sum_s[0][tid + k * per * chunks], y = sum_s[1][tid + k * per * chunks];
      acc[0] += x.x;
      acc[1] += x.y;
      acc[2] += x.z;
      acc[3] += x.w;
      acc[4] += y.x;
      acc[5] += y.y;
      acc[6] += y.z;
      acc[7] += y.w;
    }
  }
  if (!have) return;
  const int node = (first + row0 + r) / p.G, g = first + row0 + r - node * p.G;
  *reinterpret_cast<uint4 *>(p.out + (((int64_t)q * p.N + node) * p.Hq + h * p.G + g) * p.cv.D + ch * 8) = pack8<T>(acc);
}

template <typename T, int DP, bool E4M3>
cudaError_t launch_shape(const AttentionLaunch &A, const Params &p, int n_cta, cudaStream_t stream) {
  using SH = Shape<DP, E4M3>;
  static_assert(SH::SMEM <= 232448, "shared memory of one CTA");
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};  // devices this kernel is set up on
  if (dev > 63 || !((ready.load(std::memory_order_relaxed) >> dev) & 1u)) {
    if ((e = cudaFuncSetAttribute(attention_kernel<T, DP, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::SMEM)) !=
        cudaSuccess)
      return e;
    if (dev < 64) ready.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_cta);
  cfg.blockDim = dim3(SH::THREADS);
  cfg.dynamicSmemBytes = SH::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attention_kernel<T, DP, E4M3>, *A.map_k, *A.map_v, p);
  if (e != cudaSuccess || (e = cudaGetLastError()) != cudaSuccess) return e;
  // the join launches while the last CTAs run and waits for them before it reads their parts
  cfg.gridDim = dim3(n_cta, (p.part_rows + JOIN_ROWS - 1) / JOIN_ROWS);
  cfg.blockDim = dim3(JOIN_ROWS * (p.cv.D / 8));
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, join_kernel<T, SH::NS>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
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
  return (size_t)2 * ATTENTION_MAX_CTAS * part_rows(M, D) * ((size_t)D * 4 + 8) + ATTENTION_MAX_CTAS * sizeof(Cut);
}
int attention_box_rows(int page_size) {
  return page_size < BN ? page_size : BN;
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
  p.c = A.scale * ATTENTION_LOG2E;
  p.out = static_cast<uint16_t *>(A.out);
  p.lse = A.lse;
  p.status = A.status;
  p.part_rows = part_rows(p.M, A.cache.D);
  p.part_o = static_cast<float4 *>(A.ws);
  p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(A.ws) +
                                         (size_t)2 * ATTENTION_MAX_CTAS * p.part_rows * A.cache.D * 4);
  p.cuts = reinterpret_cast<Cut *>(p.part_ml + (size_t)2 * ATTENTION_MAX_CTAS * p.part_rows);
  const int n_cta = A.n_sm < ATTENTION_MAX_CTAS ? A.n_sm : ATTENTION_MAX_CTAS;
  const bool e4m3 = A.cache.dtype == MFD_E4M3;
  if (A.dtype == MFD_BF16)
    return e4m3 ? launch_width<__nv_bfloat16, true>(A, p, n_cta, stream)
                : launch_width<__nv_bfloat16, false>(A, p, n_cta, stream);
  return e4m3 ? launch_width<__half, true>(A, p, n_cta, stream) : launch_width<__half, false>(A, p, n_cta, stream);
}

}  // namespace mfd
