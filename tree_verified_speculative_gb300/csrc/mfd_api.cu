// mfd_api.cu -- the extern "C" entry points of libmfd (declared and
// documented in include/mfd.h): argument checks, scratch layout, TMA
// descriptor encoding, kernel launches.  No allocation, no host sync.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>

#include "../../include/mfd.h"
#include "delta.h"
#include "kvcache.h"
#include "lmhead.h"

namespace {

struct DeviceInfo {
  int n_sm = 0, major = 0, minor = 0;
  bool ok = false;
};

std::mutex g_mu;
std::map<int, DeviceInfo> g_dev;

int current_device_info(DeviceInfo *out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MFD_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_dev.find(dev);
  if (it == g_dev.end()) {
    DeviceInfo d;
    if (cudaDeviceGetAttribute(&d.n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return MFD_ERR_CUDA;
    d.ok = true;
    it = g_dev.emplace(dev, d).first;
  }
  *out = it->second;
  return MFD_OK;
}

bool is_sm103(const DeviceInfo &d) { return d.major == 10 && d.minor == 3; }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int cand_width(int topk) { return topk <= 8 ? 8 : (topk <= 16 ? 16 : 32); }

// ---------------------------------------------------------------- TMA maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

using MapKey = std::tuple<int, const void *, int, int, int, int, size_t>;  // device, ptr, rows, cols, box rows, bytes/elem, row stride
std::map<MapKey, CUtensorMap> g_maps;

// bf16 (elem = 2) or 8-bit (elem = 1) [rows][cols] row-major, rows `stride`
// bytes apart (0: cols * elem), box = 128 bytes of columns x box_rows rows,
// 128B swizzle, out-of-range rows read as zero.  The descriptor is copied
// into *out while the lock is held: another thread may clear the cache right
// after.
int tensor_map(const void *ptr, int rows, int cols, int box_rows, CUtensorMap *out, int elem = 2, size_t stride = 0) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MFD_ERR_CUDA;
  if (stride == 0) stride = (size_t)cols * (size_t)elem;
  std::lock_guard<std::mutex> lk(g_mu);
  const MapKey key{dev, ptr, rows, cols, box_rows, elem, stride};
  auto it = g_maps.find(key);
  if (it == g_maps.end()) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return MFD_ERR_CUDA;
    CUtensorMap m;
    std::memset(&m, 0, sizeof m);
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / elem), (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1u, 1u};
    const CUresult r = fn(&m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                          const_cast<void *>(ptr), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return MFD_ERR_CUDA;
    if (g_maps.size() > 4096) g_maps.clear();
    it = g_maps.emplace(key, m).first;
  }
  *out = it->second;
  return MFD_OK;
}

// ---------------------------------------------------------------- layouts
struct TopkLayout {
  int P, T, chunk;
  size_t ms_bytes, cand_bytes, total;
  size_t stage_off = 0;  // LM head: room for the staged hidden rows (lmhead_hidden_stage)
  size_t part_off = 0;   // LM head: the partials follow the row bound, which starts the scratch
};

// Fewest weight tiles for the busiest CTA when n_groups M tiles share
// `workers` CTAs: over P vocabulary ranges, a CTA takes
// ceil(n_groups * P / workers) items of ceil(tiles / P) tiles.  Among equal
// costs the fewest ranges win: fewer partials to merge and fewer top-T
// restarts per row.
static long long best_ranges(int tiles, int n_groups, int workers, int *P_out) {
  long long best = -1;
  const int pmax = tiles < 256 ? tiles : 256;
  for (int P = 1; P <= pmax; ++P) {
    const long long rounds = ((long long)n_groups * P + workers - 1) / workers;
    const long long cost = rounds * ((tiles + P - 1) / P);
    if (best < 0 || cost < best) {
      best = cost;
      *P_out = P;
    }
  }
  return best;
}

TopkLayout lmhead_layout(int R, int V, int topk, int n_sm) {
  TopkLayout y;
  const int tile_rows = mfd::lmhead_tile_rows(R, V, n_sm);
  const int tiles = (V + tile_rows - 1) / tile_rows;
  const int n_mt = (R + mfd::lmhead_m_rows() - 1) / mfd::lmhead_m_rows();
  y.P = tiles < n_sm ? tiles : n_sm;
  if (y.P > 256) y.P = 256;
  if (n_mt > 1) {
    best_ranges(tiles, n_mt, n_sm, &y.P);  // work items are (range, M tile)
  } else {
    // When at most three quarters of the ranges hold the largest share, the
    // last wave leaves many SMs idle: take the fewest ranges with the same
    // largest range instead, so that every CTA that streams streams as many
    // tiles (measured: 65,536 rows 64.2 -> 61.5 us, 248,320 rows at H = 5120
    // 384 -> 377 us; with 151,936 rows, 138 of 152 ranges hold four tiles,
    // and 149 ranges were slower)
    const int most = (tiles + y.P - 1) / y.P;
    const int at_most = tiles - (most - 1) * y.P;  // ranges holding `most` tiles
    if (4 * at_most <= 3 * y.P) y.P = (tiles + most - 1) / most;
  }
  y.T = cand_width(topk);
  y.chunk = 0;
  // the row bound's generation words sit at offset 0 for every shape, so a
  // call of another shape finds them where the last one left them
  y.part_off = mfd::lmhead_bound_bytes(R, y.T);
  y.ms_bytes = align256((size_t)R * y.P * 8);
  y.cand_bytes = align256((size_t)R * y.P * y.T * 8);
  y.total = y.part_off + y.ms_bytes + y.cand_bytes;
  // one M tile: room for the hidden rows staged when they span few bytes
  y.stage_off = y.total;
  if (R <= mfd::lmhead_m_rows()) y.total += align256(mfd::lmhead_stage_max_bytes());
  return y;
}

// FP8 LM head scratch: the partials of lmhead_layout, then the E4M3 hidden
// rows (R rows of H bytes, or the padded rows of lmhead_hidden_stage) and
// their scales [R].
struct Fp8Layout {
  TopkLayout y;
  size_t hq_off, sc_off, total;
};
Fp8Layout fp8_layout(int R, int H, int V, int topk, int n_sm) {
  Fp8Layout f;
  f.y = lmhead_layout(R, V, topk, n_sm);
  f.hq_off = f.y.total;
  const mfd::HiddenStage hs = mfd::lmhead_hidden_stage(R, (size_t)H);
  f.sc_off = f.hq_off + align256(hs.staged ? hs.bytes : (size_t)R * H);
  f.total = f.sc_off + align256((size_t)R * 4);
  return f;
}

TopkLayout logits_layout(int R, int V, int topk) {
  TopkLayout y;
  int chunk = (V + 255) / 256;
  chunk = (chunk + 31) / 32 * 32;
  if (chunk < 1024) chunk = 1024;
  y.chunk = chunk;
  y.P = (V + chunk - 1) / chunk;
  y.T = cand_width(topk);
  y.ms_bytes = align256((size_t)R * y.P * 8);
  y.cand_bytes = align256((size_t)R * y.P * y.T * 8);
  y.total = y.ms_bytes + y.cand_bytes;
  return y;
}

size_t verify_bytes(int n_sm) { return align256((size_t)mfd::verify_max_grid(n_sm) * 8 * 8); }

size_t analytics_bytes(int n_req, int B) { return align256((size_t)n_req * (B + 1) * 8) + align256((size_t)n_req * (B + 1) * 4); }

size_t tree_bytes(int n_req) {
  (void)n_req;
  return 256;  // the tree is built in shared memory; the scratch is not used
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? MFD_OK : MFD_ERR_CUDA; }

// Scratch of mfd_logits_topk_noalloc: one static array per device, kept
// for the life of the process.  Host code cannot use its name as a device
// address, so its address is looked up once per device.
static __device__ __align__(256) unsigned char g_noalloc_scratch[MFD_NOALLOC_SCRATCH_BYTES];

std::mutex g_noalloc_mu;
std::map<int, void *> g_noalloc_ptr;

int noalloc_scratch(void **out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MFD_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_noalloc_mu);
  auto it = g_noalloc_ptr.find(dev);
  if (it == g_noalloc_ptr.end()) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr) return MFD_ERR_CUDA;
    it = g_noalloc_ptr.emplace(dev, p).first;
  }
  *out = it->second;
  return MFD_OK;
}

}  // namespace

extern "C" {

const char *mfd_status_string(int status) {
  switch (status) {
    case MFD_OK: return "ok";
    case MFD_ERR_INVALID_ARG: return "invalid argument (NULL pointer, size out of range or misaligned pointer)";
    case MFD_ERR_UNSUPPORTED: return "unsupported: outside the library limits or not an sm_103a device";
    case MFD_ERR_WORKSPACE: return "workspace missing or smaller than mfd_workspace_size";
    case MFD_ERR_CUDA: return "a CUDA runtime or driver call failed";
    case MFD_ERR_TIMEOUT: return "a bounded device wait ran out; the kernel stopped early";
    case MFD_ERR_INPUT: return "input values break the contract (see mfd.h)";
    case MFD_ERR_CHECK: return "bounds-checked build: an index out of range was clamped";
    default: return "unknown status";
  }
}

int mfd_tree_analytics(const int32_t *parent, const int32_t *token, const int32_t *depth, const int32_t *n_nodes,
                       int n_req, int B, int L, const int32_t *futures, int F, const float *target_logits, int V,
                       const float *temperature, int32_t *node_class, double *reach, double *mass, int32_t *status,
                       void *ws, size_t ws_bytes, mfd_stream_t stream) {
  if (!parent || !token || !depth || !n_nodes || !futures || !target_logits || !temperature || !node_class ||
      !reach || !mass || !status)
    return MFD_ERR_INVALID_ARG;
  if (n_req < 1 || B < 1 || L < 1 || F < 1 || V < 1) return MFD_ERR_INVALID_ARG;
  if (B > 512 || L > 16 || F > 64 || V >= (1 << 30)) return MFD_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < analytics_bytes(n_req, B) || !aligned(ws, 256)) return MFD_ERR_WORKSPACE;
  char *base = static_cast<char *>(ws);
  mfd::AnalyticsLaunch A;
  A.t = target_logits;
  A.n_req = n_req;
  A.B = B;
  A.V = V;
  A.L = L;
  A.parent = parent;
  A.token = token;
  A.depth = depth;
  A.n_nodes = n_nodes;
  A.futures = futures;
  A.F = F;
  A.temperature = temperature;
  A.lse = reinterpret_cast<double *>(base);
  A.amax = reinterpret_cast<int32_t *>(base + align256((size_t)n_req * (B + 1) * 8));
  A.node_class = node_class;
  A.reach = reach;
  A.mass = mass;
  A.status = status;
  return cuda_status(mfd::launch_tree_analytics(A, reinterpret_cast<cudaStream_t>(stream)));
}

int mfd_mfdd_modes(int n_req, int K) {
  if (n_req < 1 || K < 1 || K > 16) return 0;
  return n_req < MFD_MFDD_SWITCH_REQUESTS ? K : 1;
}

size_t mfd_workspace_size(int op, int n_req, int K, int L, int topk, int B, int R, int V) {
  (void)K;
  (void)L;
  (void)B;
  DeviceInfo d;
  switch (op) {
    case MFD_OP_LMHEAD_TOPK:
      if (R < 1 || V < 16 || topk < 1 || topk > 32 || topk > V) return 0;
      if (current_device_info(&d) != MFD_OK) return 0;
      return lmhead_layout(R, V, topk, d.n_sm).total;
    case MFD_OP_LOGITS_TOPK:
      if (R < 1 || V < 16 || topk < 1 || topk > 32 || topk > V) return 0;
      return logits_layout(R, V, topk).total;
    case MFD_OP_BUILD_TREE:
      if (n_req < 1) return 0;
      return tree_bytes(n_req);
    case MFD_OP_VERIFY:
      if (n_req < 1) return 0;
      if (current_device_info(&d) != MFD_OK) return 0;
      return verify_bytes(d.n_sm);
    case MFD_OP_TREE_ANALYTICS:
      if (n_req < 1 || B < 1 || B > 512) return 0;
      return analytics_bytes(n_req, B);
    default:
      return 0;
  }
}

}  // extern "C"

namespace {
// The LM head call, from the row-major weight (W, through its tensor map) or
// from the packed weight (Wp).
// vocab_ids: null, or the draft-vocabulary subset (V rows of the weight are
// vocabulary ids vocab_ids[0..V), increasing, below V_full)
int lmhead_call(const void *h, int R, int H, const void *W, const void *Wp, int V, int topk, float *tk_logp,
                int32_t *tk_tok, float *lse, int32_t *status, void *ws, size_t ws_bytes, mfd_stream_t stream,
                const int32_t *vocab_ids = nullptr, int V_full = 0, bool fp8 = false, bool withhold = false) {
  if (!h || (!W && !Wp) || !tk_logp || !tk_tok || !status || R < 1 || H < 1 || V < 1 || topk < 1)
    return MFD_ERR_INVALID_ARG;
  if (!aligned(h, 16) || (W && !aligned(W, 16)) || (Wp && !aligned(Wp, 256))) return MFD_ERR_INVALID_ARG;
  if (H % ((fp8 ? 2 : 1) * mfd::lmhead_k_chunk()) != 0 || topk > 32 || V < 16 || topk > V || V >= (1 << 30))
    return MFD_ERR_UNSUPPORTED;
  DeviceInfo d;
  int rc = current_device_info(&d);
  if (rc != MFD_OK) return rc;
  if (!is_sm103(d)) return MFD_ERR_UNSUPPORTED;
  const TopkLayout y = lmhead_layout(R, V, topk, d.n_sm);
  const Fp8Layout f8 = fp8_layout(R, H, V, topk, d.n_sm);
  if (!ws || ws_bytes < (fp8 ? f8.total : y.total) || !aligned(ws, 256)) return MFD_ERR_WORKSPACE;
  char *base = static_cast<char *>(ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CUtensorMap mh, mw;
  // hidden rows that span few bytes are read from a padded copy
  const mfd::HiddenStage hs = mfd::lmhead_hidden_stage(R, (size_t)H * (fp8 ? 1 : 2));
  if (fp8) {
    // the hidden rows in E4M3 with their scales, then the E4M3 head over them
    if ((rc = cuda_status(mfd::launch_quant_rows(h, R, H, base + f8.hq_off, reinterpret_cast<float *>(base + f8.sc_off),
                                                 s, hs.rows, hs.stride))) != MFD_OK)
      return rc;
    if ((rc = tensor_map(base + f8.hq_off, hs.rows, H, mfd::lmhead_m_rows(), &mh, 1, hs.stride)) != MFD_OK) return rc;
  } else if (hs.staged) {
    char *hstage = base + y.stage_off;
    if ((rc = cuda_status(mfd::launch_stage_rows(h, R, (size_t)H * 2, hstage, hs, s))) != MFD_OK) return rc;
    if ((rc = tensor_map(hstage, hs.rows, H, mfd::lmhead_m_rows(), &mh, 2, hs.stride)) != MFD_OK) return rc;
  } else if ((rc = tensor_map(h, R, H, mfd::lmhead_m_rows(), &mh)) != MFD_OK) {
    return rc;
  }
  if (W && (rc = tensor_map(W, V, H, mfd::lmhead_tile_rows(R, V, d.n_sm), &mw)) != MFD_OK) return rc;
  mfd::LmheadLaunch L;
  L.tmap_h = &mh;
  L.tmap_w = W ? &mw : nullptr;
  L.w_packed = W ? nullptr : Wp;
  L.R = R;
  L.H = H;
  L.V = V;
  L.T = y.T;
  L.P = y.P;
  L.n_sm = d.n_sm;
  L.tile_rows = mfd::lmhead_tile_rows(R, V, d.n_sm);
  L.part_ms = base + y.part_off;
  L.part_cand = base + y.part_off + y.ms_bytes;
  L.status = status;
  L.withhold = withhold;
  L.rb = y.part_off ? base : nullptr;
  L.G = topk;
  if (fp8) {
    L.fp8 = true;
    L.row_scale = reinterpret_cast<const float *>(base + f8.sc_off);
    L.w_amax = reinterpret_cast<const float *>(static_cast<const char *>(Wp) + mfd::lmhead_packed_fp8_bytes(V, H) - 256);
  }
  if ((rc = cuda_status(mfd::launch_lmhead_partials(L, s))) != MFD_OK) return rc;
  mfd::MergeLaunch M;
  M.part_ms = L.part_ms;
  M.part_cand = L.part_cand;
  M.R = R;
  M.P = y.P;
  M.T = y.T;
  M.topk = topk;
  M.tk_logp = tk_logp;
  M.tk_tok = tk_tok;
  M.lse = lse;
  M.status = status;
  M.vocab_ids = vocab_ids;
  M.V_sub = V;
  M.V_full = vocab_ids ? V_full : V;
  M.rb = L.rb ? reinterpret_cast<const int *>(base + mfd::LMHEAD_BOUND_HEADER) : nullptr;
  M.G = topk;
  return cuda_status(mfd::launch_merge_topk(M, s));
}
}  // namespace

extern "C" {

int mfd_lmhead_topk(const void *h, int R, int H, const void *W, int V, int topk, float *tk_logp,
                    int32_t *tk_tok, float *lse, int32_t *status, void *ws, size_t ws_bytes,
                    mfd_stream_t stream) {
  if (!W) return MFD_ERR_INVALID_ARG;
  return lmhead_call(h, R, H, W, nullptr, V, topk, tk_logp, tk_tok, lse, status, ws, ws_bytes, stream);
}

size_t mfd_lmhead_packed_bytes(int V, int H) {
  if (V < 16 || V >= (1 << 30) || H < 1 || H % mfd::lmhead_k_chunk() != 0) return 0;
  return mfd::lmhead_packed_bytes(V, H);
}

int mfd_lmhead_pack(const void *W, int V, int H, void *W_packed, size_t packed_bytes, mfd_stream_t stream) {
  if (!W || !W_packed || V < 1 || H < 1) return MFD_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(W_packed, 256)) return MFD_ERR_INVALID_ARG;
  const size_t need = mfd_lmhead_packed_bytes(V, H);
  if (need == 0) return MFD_ERR_UNSUPPORTED;
  if (packed_bytes < need) return MFD_ERR_WORKSPACE;
  DeviceInfo d;
  int rc = current_device_info(&d);
  if (rc != MFD_OK) return rc;
  if (!is_sm103(d)) return MFD_ERR_UNSUPPORTED;
  return cuda_status(mfd::launch_pack_w(W, V, H, W_packed, reinterpret_cast<cudaStream_t>(stream)));
}

int mfd_lmhead_topk_packed(const void *h, int R, int H, const void *W_packed, int V, int topk, float *tk_logp,
                           int32_t *tk_tok, float *lse, int32_t *status, void *ws, size_t ws_bytes,
                           mfd_stream_t stream) {
  if (!W_packed) return MFD_ERR_INVALID_ARG;
  return lmhead_call(h, R, H, nullptr, W_packed, V, topk, tk_logp, tk_tok, lse, status, ws, ws_bytes, stream);
}

int mfd_lmhead_withheld_test(const void *h, int R, int H, const void *W_packed, int V, int topk, float *tk_logp,
                             int32_t *tk_tok, float *lse, int32_t *status, void *ws, size_t ws_bytes,
                             mfd_stream_t stream) {
  if (!W_packed) return MFD_ERR_INVALID_ARG;
  return lmhead_call(h, R, H, nullptr, W_packed, V, topk, tk_logp, tk_tok, lse, status, ws, ws_bytes, stream,
                     nullptr, 0, false, true);
}

size_t mfd_lmhead_packed_fp8_bytes(int V, int H) {
  if (V < 16 || V >= (1 << 30) || H < 1 || H % (2 * mfd::lmhead_k_chunk()) != 0) return 0;
  return mfd::lmhead_packed_fp8_bytes(V, H);
}

int mfd_lmhead_pack_fp8(const void *W, int V, int H, void *W_packed, size_t packed_bytes, mfd_stream_t stream) {
  if (!W || !W_packed || V < 1 || H < 1) return MFD_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(W_packed, 256)) return MFD_ERR_INVALID_ARG;
  const size_t need = mfd_lmhead_packed_fp8_bytes(V, H);
  if (need == 0) return MFD_ERR_UNSUPPORTED;
  if (packed_bytes < need) return MFD_ERR_WORKSPACE;
  DeviceInfo d;
  int rc = current_device_info(&d);
  if (rc != MFD_OK) return rc;
  if (!is_sm103(d)) return MFD_ERR_UNSUPPORTED;
  return cuda_status(mfd::launch_pack_w_fp8(W, V, H, W_packed, reinterpret_cast<cudaStream_t>(stream)));
}

int mfd_fp8_quantize_rows(const void *x, int R, int H, void *q, float *scale, mfd_stream_t stream) {
  if (!x || !q || !scale || R < 1 || H < 8 || H % 8 != 0) return MFD_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 8) || !aligned(scale, 4)) return MFD_ERR_INVALID_ARG;
  DeviceInfo d;
  int rc = current_device_info(&d);
  if (rc != MFD_OK) return rc;
  if (!is_sm103(d)) return MFD_ERR_UNSUPPORTED;
  return cuda_status(mfd::launch_quant_rows(x, R, H, q, scale, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mfd_lmhead_fp8_workspace_bytes(int R, int H, int V, int topk) {
  if (R < 1 || H < 1 || H % (2 * mfd::lmhead_k_chunk()) != 0 || V < 16 || topk < 1 || topk > 32 || topk > V)
    return 0;
  DeviceInfo d;
  if (current_device_info(&d) != MFD_OK) return 0;
  return fp8_layout(R, H, V, topk, d.n_sm).total;
}

int mfd_lmhead_topk_fp8(const void *h, int R, int H, const void *W_packed_fp8, int V, int topk, float *tk_logp,
                        int32_t *tk_tok, float *lse, int32_t *status, void *ws, size_t ws_bytes,
                        mfd_stream_t stream) {
  if (!W_packed_fp8) return MFD_ERR_INVALID_ARG;
  return lmhead_call(h, R, H, nullptr, W_packed_fp8, V, topk, tk_logp, tk_tok, lse, status, ws, ws_bytes, stream,
                     nullptr, 0, true);
}

int mfd_lmhead_topk_subset(const void *h, int R, int H, const void *W_packed, int V_sub, const int32_t *vocab_ids,
                           int V_full, int topk, float *tk_logp, int32_t *tk_tok, float *lse, int32_t *status,
                           void *ws, size_t ws_bytes, mfd_stream_t stream) {
  if (!W_packed || !vocab_ids || !aligned(vocab_ids, 4)) return MFD_ERR_INVALID_ARG;
  if (V_full < V_sub || V_full >= (1 << 30)) return MFD_ERR_INVALID_ARG;
  return lmhead_call(h, R, H, nullptr, W_packed, V_sub, topk, tk_logp, tk_tok, lse, status, ws, ws_bytes, stream,
                     vocab_ids, V_full);
}

int mfd_logits_topk(const float *logits, int R, int V, int topk, float *tk_logp, int32_t *tk_tok, float *lse,
                    int32_t *status, void *ws, size_t ws_bytes, mfd_stream_t stream) {
  if (!logits || !tk_logp || !tk_tok || !status || R < 1 || V < 1 || topk < 1) return MFD_ERR_INVALID_ARG;
  if (topk > 32 || V < 16 || topk > V || V >= (1 << 30)) return MFD_ERR_UNSUPPORTED;
  const TopkLayout y = logits_layout(R, V, topk);
  if (!ws || ws_bytes < y.total || !aligned(ws, 256)) return MFD_ERR_WORKSPACE;
  char *base = static_cast<char *>(ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  mfd::LogitsPartialLaunch L;
  L.logits = logits;
  L.R = R;
  L.V = V;
  L.T = y.T;
  L.P = y.P;
  L.chunk = y.chunk;
  L.part_ms = base;
  L.part_cand = base + y.ms_bytes;
  int rc = cuda_status(mfd::launch_logits_partials(L, s));
  if (rc != MFD_OK) return rc;
  mfd::MergeLaunch M;
  M.part_ms = L.part_ms;
  M.part_cand = L.part_cand;
  M.R = R;
  M.P = y.P;
  M.T = y.T;
  M.topk = topk;
  M.tk_logp = tk_logp;
  M.tk_tok = tk_tok;
  M.lse = lse;
  M.status = status;
  M.vocab_ids = nullptr;
  M.V_sub = M.V_full = V;
  return cuda_status(mfd::launch_merge_topk(M, s));
}

int mfd_logits_topk_noalloc(const float *logits, int R, int V, int topk, float *tk_logp, int32_t *tk_tok,
                            float *lse, int32_t *status, mfd_stream_t stream) {
  if (!logits || !tk_logp || !tk_tok || !status || R < 1 || V < 1 || topk < 1) return MFD_ERR_INVALID_ARG;
  if (topk > 32 || V < 16 || topk > V || V >= (1 << 30)) return MFD_ERR_UNSUPPORTED;
  const TopkLayout y = logits_layout(R, V, topk);
  if (y.total > MFD_NOALLOC_SCRATCH_BYTES) return MFD_ERR_WORKSPACE;  // too large for the fixed scratch
  void *scratch = nullptr;
  int rc = noalloc_scratch(&scratch);
  if (rc != MFD_OK) return rc;
  char *base = static_cast<char *>(scratch);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  mfd::LogitsPartialLaunch L;
  L.logits = logits;
  L.R = R;
  L.V = V;
  L.T = y.T;
  L.P = y.P;
  L.chunk = y.chunk;
  L.part_ms = base;
  L.part_cand = base + y.ms_bytes;
  rc = cuda_status(mfd::launch_logits_partials(L, s));
  if (rc != MFD_OK) return rc;
  mfd::MergeLaunch M;
  M.part_ms = L.part_ms;
  M.part_cand = L.part_cand;
  M.R = R;
  M.P = y.P;
  M.T = y.T;
  M.topk = topk;
  M.tk_logp = tk_logp;
  M.tk_tok = tk_tok;
  M.lse = lse;
  M.status = status;
  M.vocab_ids = nullptr;
  M.V_sub = M.V_full = V;
  return cuda_status(mfd::launch_merge_topk(M, s));
}

int mfd_build_tree(const float *tk_logp, const int32_t *tk_tok, int n_req, int K, int L, int topk, int B,
                   const int32_t *anchor_tok, const int32_t *base_pos, int32_t *parent, int32_t *token,
                   int32_t *depth, float *score, int32_t *mode, uint32_t *mask, int32_t *pos, int32_t *n_nodes,
                   int32_t *status, void *ws, size_t ws_bytes, mfd_stream_t stream) {
  if (!tk_logp || !tk_tok || !anchor_tok || !parent || !token || !depth || !score || !mode || !mask || !pos ||
      !n_nodes || !status)
    return MFD_ERR_INVALID_ARG;
  if (n_req < 1 || K < 1 || L < 1 || topk < 1 || B < 1) return MFD_ERR_INVALID_ARG;
  if (K > 16 || L > 16 || topk > 32 || B > 512 || K * B > 2048) return MFD_ERR_UNSUPPORTED;
  int cap = 0, tsize = 0;
  if (mfd::tree_smem_bytes(K, L, topk, B, &cap, &tsize) == 0) return MFD_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < tree_bytes(n_req) || !aligned(ws, 256)) return MFD_ERR_WORKSPACE;
  mfd::TreeLaunch T;
  T.tk_logp = tk_logp;
  T.tk_tok = tk_tok;
  T.n_req = n_req;
  T.K = K;
  T.L = L;
  T.topk = topk;
  T.B = B;
  T.anchor = anchor_tok;
  T.base_pos = base_pos;
  T.parent = parent;
  T.token = token;
  T.depth = depth;
  T.score = score;
  T.mode = mode;
  T.mask = mask;
  T.pos = pos;
  T.n_nodes = n_nodes;
  T.status = status;
  return cuda_status(mfd::launch_build_tree(T, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {
int verify_call(const float *target_logits, int n_req, int B, int V, int L, const int32_t *parent,
                const int32_t *token, const int32_t *n_nodes, const float *temperature, const uint64_t *seed,
                int32_t *accept_len, int32_t *path_nodes, int32_t *out_tokens, int32_t *status, void *ws,
                size_t ws_bytes, mfd_stream_t stream, unsigned long long wait_ns, int withhold) {
  if (!target_logits || !parent || !token || !n_nodes || !temperature || !seed || !accept_len || !path_nodes ||
      !out_tokens || !status)
    return MFD_ERR_INVALID_ARG;
  if (n_req < 1 || B < 1 || V < 2 || L < 1) return MFD_ERR_INVALID_ARG;
  if (B > 512 || L > 16 || V >= (1 << 30)) return MFD_ERR_UNSUPPORTED;
  DeviceInfo d;
  int rc = current_device_info(&d);
  if (rc != MFD_OK) return rc;
  if (!ws || ws_bytes < verify_bytes(d.n_sm) || !aligned(ws, 256)) return MFD_ERR_WORKSPACE;
  // the target logits: device memory, or page-locked host memory mapped into
  // the device's address space, which the walk reads in place (only the rows
  // on the walk cross the host link)
  cudaPointerAttributes pa;
  if (cudaPointerGetAttributes(&pa, target_logits) != cudaSuccess) {
    (void)cudaGetLastError();
    return MFD_ERR_INVALID_ARG;
  }
  const float *t = target_logits;
  if (pa.type == cudaMemoryTypeHost) {
    if (!pa.devicePointer) return MFD_ERR_INVALID_ARG;
    t = static_cast<const float *>(pa.devicePointer);
  } else if (pa.type != cudaMemoryTypeDevice && pa.type != cudaMemoryTypeManaged) {
    return MFD_ERR_INVALID_ARG;  // pageable host memory
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  mfd::VerifyLaunch Vl;
  Vl.t = t;
  Vl.n_req = n_req;
  Vl.B = B;
  Vl.V = V;
  Vl.L = L;
  Vl.parent = parent;
  Vl.token = token;
  Vl.n_nodes = n_nodes;
  Vl.temperature = temperature;
  Vl.seed = seed;
  Vl.accept_len = accept_len;
  Vl.path_nodes = path_nodes;
  Vl.out_tokens = out_tokens;
  Vl.status = status;
  Vl.ws = static_cast<unsigned long long *>(ws);
  Vl.grid = mfd::verify_max_grid(d.n_sm);
  Vl.wait_ns = wait_ns;
  Vl.withhold = withhold;
  return cuda_status(mfd::launch_verify(Vl, s));
}
}  // namespace

extern "C" {

int mfd_verify(const float *target_logits, int n_req, int B, int V, int L, const int32_t *parent,
               const int32_t *token, const int32_t *n_nodes, const float *temperature, const uint64_t *seed,
               int32_t *accept_len, int32_t *path_nodes, int32_t *out_tokens, int32_t *status, void *ws,
               size_t ws_bytes, mfd_stream_t stream) {
  return verify_call(target_logits, n_req, B, V, L, parent, token, n_nodes, temperature, seed, accept_len,
                     path_nodes, out_tokens, status, ws, ws_bytes, stream, 0ull, 0);
}

int mfd_verify_withheld_test(const float *target_logits, int n_req, int B, int V, int L, const int32_t *parent,
                             const int32_t *token, const int32_t *n_nodes, const float *temperature,
                             const uint64_t *seed, int32_t *accept_len, int32_t *path_nodes, int32_t *out_tokens,
                             int32_t *status, void *ws, size_t ws_bytes, uint64_t wait_limit_ns,
                             mfd_stream_t stream) {
  if (wait_limit_ns < 1000ull || wait_limit_ns > 100000000ull) return MFD_ERR_INVALID_ARG;
  return verify_call(target_logits, n_req, B, V, L, parent, token, n_nodes, temperature, seed, accept_len,
                     path_nodes, out_tokens, status, ws, ws_bytes, stream, wait_limit_ns, 1);
}

}  // extern "C"

// ------------------------------------------- attention over a paged cache
namespace {

// mfd_kv_cache to the kernels' view, with its limits checked.
int cache_view(const mfd_kv_cache *c, mfd::CacheView *out) {
  if (!c || !c->k || !c->v || !c->block_table) return MFD_ERR_INVALID_ARG;
  if (c->dtype != MFD_BF16 && c->dtype != MFD_FP16 && c->dtype != MFD_E4M3) return MFD_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->Hk < 1 || c->D < 1) return MFD_ERR_INVALID_ARG;
  const bool e4m3 = c->dtype == MFD_E4M3;
  if (e4m3 && (!c->k_exp || !c->v_exp)) return MFD_ERR_INVALID_ARG;
  const int64_t esz = e4m3 ? 1 : 2;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->block_table, 4)) return MFD_ERR_INVALID_ARG;
  if (c->D % 16 != 0 || c->D > 256 || c->Hk > 1024) return MFD_ERR_UNSUPPORTED;
  const int64_t strides[3] = {c->page_stride, c->head_stride, c->token_stride};
  for (int64_t s : strides) {
    if (s < c->D || s * esz % 16 != 0) return MFD_ERR_INVALID_ARG;
    if (s * esz >= ((int64_t)1 << 40)) return MFD_ERR_UNSUPPORTED;  // a tensor map's stride
  }
  int shift = 4;
  while (shift < 8 && (1 << shift) < c->page_size) ++shift;
  if ((1 << shift) != c->page_size) return MFD_ERR_UNSUPPORTED;
  if ((int64_t)c->max_pages * c->page_size >= ((int64_t)1 << 31) - 65536) return MFD_ERR_UNSUPPORTED;
  out->k = c->k;
  out->v = c->v;
  out->k_exp = e4m3 ? c->k_exp : nullptr;
  out->v_exp = e4m3 ? c->v_exp : nullptr;
  out->table = c->block_table;
  out->dtype = c->dtype;
  out->n_pages = c->n_pages;
  out->ps_shift = shift;
  out->max_pages = c->max_pages;
  out->Hk = c->Hk;
  out->D = c->D;
  out->page_stride = c->page_stride;
  out->head_stride = c->head_stride;
  out->token_stride = c->token_stride;
  return MFD_OK;
}

// Keys or values as a 4-D tensor (D, slot, head, page).  A 16-bit cache's box
// is 64 columns x `rows` slots of one head and page with the 128-byte swizzle
// (columns past D read as zero); an E4M3 one's is D or 128 columns x `rows`
// slots as they are.
int kv_map(const void *ptr, const mfd::CacheView &c, int rows, CUtensorMap *out) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return MFD_ERR_CUDA;
  const bool e4m3 = c.dtype == MFD_E4M3;
  const int esz = e4m3 ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)1 << c.ps_shift, (cuuint64_t)c.Hk, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)(c.token_stride * esz), (cuuint64_t)(c.head_stride * esz),
                                 (cuuint64_t)(c.page_stride * esz)};
  const cuuint32_t box[4] = {(cuuint32_t)(!e4m3 ? 64 : c.D < 128 ? c.D : 128), (cuuint32_t)rows, 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  const CUresult r = fn(out, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : c.dtype == MFD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        4, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MFD_OK : MFD_ERR_CUDA;
}

int need_sm103() {
  DeviceInfo d;
  const int rc = current_device_info(&d);
  if (rc != MFD_OK) return rc;
  return is_sm103(d) ? MFD_OK : MFD_ERR_UNSUPPORTED;
}

// A [tokens][heads][D] tensor of 16-bit elements with its token stride.
bool rows_ok(const void *p, int64_t stride, int heads, int D) {
  return p && aligned(p, 16) && stride >= (int64_t)heads * D && stride % 8 == 0 && stride < ((int64_t)1 << 40);
}

// What the norm and rotation of mfd_qk_norm_rope and mfd_kv_append share.
int norm_rope_args(int dtype, int D, const void *q_w, const void *k_w, float eps, const uint64_t *phase, int rot_dim,
                   const int32_t *pos, const int32_t *status) {
  if (dtype != MFD_BF16 && dtype != MFD_FP16) return MFD_ERR_INVALID_ARG;
  if (!pos || !status || D < 1) return MFD_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return MFD_ERR_INVALID_ARG;
  if ((q_w && !aligned(q_w, 16)) || (k_w && !aligned(k_w, 16))) return MFD_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0 || (rot_dim > 0 && !phase)) return MFD_ERR_INVALID_ARG;
  if (D % 16 != 0 || D > 256) return MFD_ERR_UNSUPPORTED;
  return MFD_OK;
}

}  // namespace

extern "C" {

int mfd_rope_phases(const double *inv_freq, int n, uint64_t *phase) {
  if (!inv_freq || !phase || n < 1) return MFD_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!(inv_freq[i] >= 0.0) || !std::isfinite(inv_freq[i])) return MFD_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const double turns = inv_freq[i] / 6.283185307179586476925;
    const double part = turns - std::floor(turns);  // in [0, 1), at most 1 - 2^-53
    phase[i] = static_cast<uint64_t>(std::ldexp(part, 64));
  }
  return MFD_OK;
}

int mfd_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int dtype, int T, int Hq,
                     int Hk, int D, const void *q_w, const void *k_w, float eps, const uint64_t *phase, int rot_dim,
                     int interleaved, const int32_t *pos, void *q_out, void *k_out, int32_t *status,
                     mfd_stream_t stream) {
  if (T < 1 || Hq < 1 || Hk < 1) return MFD_ERR_INVALID_ARG;
  int rc = norm_rope_args(dtype, D, q_w, k_w, eps, phase, rot_dim, pos, status);
  if (rc != MFD_OK) return rc;
  if (!rows_ok(q, q_stride, Hq, D) || !rows_ok(k, k_stride, Hk, D)) return MFD_ERR_INVALID_ARG;
  if (!q_out || !k_out || !aligned(q_out, 16) || !aligned(k_out, 16)) return MFD_ERR_INVALID_ARG;
  if (Hq > 1024 || Hk > 1024) return MFD_ERR_UNSUPPORTED;
  if ((rc = need_sm103()) != MFD_OK) return rc;
  mfd::AppendLaunch A = {};
  A.q = q;
  A.k = k;
  A.q_stride = q_stride;
  A.k_stride = k_stride;
  A.dtype = dtype;
  A.n_req = 1;
  A.N = T;
  A.Hq = Hq;
  A.Hk = Hk;
  A.D = D;
  A.q_w = q_w;
  A.k_w = k_w;
  A.eps = eps;
  A.phase = phase;
  A.rot_dim = rot_dim;
  A.interleaved = interleaved != 0;
  A.pos = pos;
  A.q_out = q_out;
  A.k_out = k_out;
  A.status = status;
  return cuda_status(mfd::launch_kv_append(A, reinterpret_cast<cudaStream_t>(stream)));
}

int mfd_kv_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                  int dtype, int n_req, int N, int Hq, const void *q_w, const void *k_w, float eps,
                  const uint64_t *phase, int rot_dim, int interleaved, const int32_t *pos, const int32_t *ctx_len,
                  const int32_t *n_nodes, void *q_out, const mfd_kv_cache *cache, int32_t *status,
                  mfd_stream_t stream) {
  mfd::CacheView cv;
  int rc = cache_view(cache, &cv);
  if (rc != MFD_OK) return rc;
  if (n_req < 1 || N < 1 || Hq < 0 || !ctx_len) return MFD_ERR_INVALID_ARG;
  if ((rc = norm_rope_args(dtype, cv.D, q_w, k_w, eps, phase, rot_dim, pos, status)) != MFD_OK) return rc;
  if (cv.dtype != dtype && cv.dtype != MFD_E4M3) return MFD_ERR_INVALID_ARG;
  if (Hq > 0 && (!rows_ok(q, q_stride, Hq, cv.D) || !q_out || !aligned(q_out, 16))) return MFD_ERR_INVALID_ARG;
  if (!rows_ok(k, k_stride, cv.Hk, cv.D) || !rows_ok(v, v_stride, cv.Hk, cv.D)) return MFD_ERR_INVALID_ARG;
  if (Hq > 1024 || (int64_t)n_req * N >= ((int64_t)1 << 31) - 1) return MFD_ERR_UNSUPPORTED;
  if ((rc = need_sm103()) != MFD_OK) return rc;
  mfd::AppendLaunch A = {};
  A.q = q;
  A.k = k;
  A.v = v;
  A.q_stride = q_stride;
  A.k_stride = k_stride;
  A.v_stride = v_stride;
  A.dtype = dtype;
  A.n_req = n_req;
  A.N = N;
  A.Hq = Hq;
  A.Hk = cv.Hk;
  A.D = cv.D;
  A.q_w = Hq ? q_w : nullptr;
  A.k_w = k_w;
  A.eps = eps;
  A.phase = phase;
  A.rot_dim = rot_dim;
  A.interleaved = interleaved != 0;
  A.pos = pos;
  A.ctx_len = ctx_len;
  A.n_nodes = n_nodes;
  A.q_out = q_out;
  A.cache = &cv;
  A.status = status;
  return cuda_status(mfd::launch_kv_append(A, reinterpret_cast<cudaStream_t>(stream)));
}

int mfd_kv_read(const mfd_kv_cache *cache, int n_req, int L_max, const int32_t *start, const int32_t *length,
                int dtype, void *k_out, void *v_out, int32_t *status, mfd_stream_t stream) {
  mfd::CacheView cv;
  int rc = cache_view(cache, &cv);
  if (rc != MFD_OK) return rc;
  if (n_req < 1 || L_max < 1 || !start || !length || !k_out || !v_out || !status) return MFD_ERR_INVALID_ARG;
  if (dtype != MFD_BF16 && dtype != MFD_FP16) return MFD_ERR_INVALID_ARG;
  if (cv.dtype != MFD_E4M3 && cv.dtype != dtype) return MFD_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return MFD_ERR_INVALID_ARG;
  if (n_req > 65535 || (int64_t)L_max * cv.Hk >= ((int64_t)1 << 33)) return MFD_ERR_UNSUPPORTED;
  if ((rc = need_sm103()) != MFD_OK) return rc;
  mfd::KvReadLaunch A;
  A.cache = cv;
  A.n_req = n_req;
  A.L_max = L_max;
  A.dtype = dtype;
  A.start = start;
  A.length = length;
  A.k_out = k_out;
  A.v_out = v_out;
  A.status = status;
  return cuda_status(mfd::launch_kv_read(A, reinterpret_cast<cudaStream_t>(stream)));
}

int mfd_kv_commit(const mfd_kv_cache *cache, int n_req, int L, const int32_t *ctx_len, const int32_t *accept_len,
                  const int32_t *path_nodes, const int32_t *n_nodes, int32_t *new_len, int32_t *status,
                  mfd_stream_t stream) {
  mfd::CacheView cv;
  int rc = cache_view(cache, &cv);
  if (rc != MFD_OK) return rc;
  if (n_req < 1 || L < 1 || !ctx_len || !accept_len || !path_nodes || !n_nodes || !new_len || !status)
    return MFD_ERR_INVALID_ARG;
  if (L > 16) return MFD_ERR_UNSUPPORTED;
  if ((rc = need_sm103()) != MFD_OK) return rc;
  mfd::KvCommitLaunch A;
  A.cache = cv;
  A.n_req = n_req;
  A.L = L;
  A.ctx_len = ctx_len;
  A.accept_len = accept_len;
  A.path = path_nodes;
  A.n_nodes = n_nodes;
  A.new_len = new_len;
  A.status = status;
  return cuda_status(mfd::launch_kv_commit(A, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mfd_tree_attention_workspace_bytes(int n_req, int N, int Hq, int Hk, int D) {
  if (n_req < 1 || n_req > 1024 || N < 1 || N > 4096 || Hq < 1 || Hk < 1 || Hq > 1024 || Hq % Hk != 0 ||
      (int64_t)N * (Hq / Hk) > 65536 || D < 16 || D > 256 || D % 16 != 0)
    return 0;
  return align256(mfd::attention_part_bytes(N * (Hq / Hk), D));
}

int mfd_tree_attention(const void *q, int64_t q_stride, int dtype, int n_req, int N, int Hq,
                       const mfd_kv_cache *cache, const int32_t *ctx_len, const int32_t *n_nodes,
                       const uint32_t *mask, float scale, void *out, float *lse, int32_t *status, void *ws,
                       size_t ws_bytes, mfd_stream_t stream) {
  mfd::CacheView cv;
  int rc = cache_view(cache, &cv);
  if (rc != MFD_OK) return rc;
  if (n_req < 1 || N < 1 || Hq < 1 || !ctx_len || !out || !status) return MFD_ERR_INVALID_ARG;
  if (dtype != MFD_BF16 && dtype != MFD_FP16) return MFD_ERR_INVALID_ARG;
  if (cv.dtype != dtype && cv.dtype != MFD_E4M3) return MFD_ERR_INVALID_ARG;
  if (!rows_ok(q, q_stride, Hq, cv.D) || !aligned(out, 16)) return MFD_ERR_INVALID_ARG;
  // the kernel works with powers of two: scale * log2 e has to be a number too
  if (!(scale > 0.f) || !std::isfinite(scale * mfd::ATTENTION_LOG2E)) return MFD_ERR_INVALID_ARG;
  const size_t need = mfd_tree_attention_workspace_bytes(n_req, N, Hq, cv.Hk, cv.D);
  if (need == 0) return MFD_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MFD_ERR_WORKSPACE;
  DeviceInfo d;
  if ((rc = current_device_info(&d)) != MFD_OK) return rc;
  if (!is_sm103(d)) return MFD_ERR_UNSUPPORTED;
  CUtensorMap mk, mv;
  const int rows = mfd::attention_box_rows(1 << cv.ps_shift);
  if ((rc = kv_map(cv.k, cv, rows, &mk)) != MFD_OK || (rc = kv_map(cv.v, cv, rows, &mv)) != MFD_OK) return rc;
  mfd::AttentionLaunch A;
  A.map_k = &mk;
  A.map_v = &mv;
  A.n_sm = d.n_sm;
  A.ws = ws;
  A.q = q;
  A.q_stride = q_stride;
  A.dtype = dtype;
  A.n_req = n_req;
  A.N = N;
  A.Hq = Hq;
  A.cache = cv;
  A.ctx_len = ctx_len;
  A.n_nodes = n_nodes;
  A.mask = mask;
  A.scale = scale;
  A.out = out;
  A.lse = lse;
  A.status = status;
  return cuda_status(mfd::launch_tree_attention(A, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// What the three forms of the delta rule share; fills A from it.
int delta_args(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int dtype, int n_req, int N, int Hk,
               const float *g, const float *beta, int normalize, float eps, const int32_t *n_nodes,
               const mfd_delta_state *state, const int32_t *src, const int32_t *dst, int32_t *status,
               mfd::DeltaArgs *A) {
  if (!state || !state->s || !aligned(state->s, 16) || state->n_slots < 1 || state->Hv < 1 || state->Dk < 1 || state->Dv < 1)
    return MFD_ERR_INVALID_ARG;
  if (dtype != MFD_BF16 && dtype != MFD_FP16) return MFD_ERR_INVALID_ARG;
  if (n_req < 1 || N < 1 || Hk < 1 || !g || !beta || !status) return MFD_ERR_INVALID_ARG;
  for (const void *a : {(const void *)g, (const void *)beta, (const void *)n_nodes, (const void *)src, (const void *)dst,
                        (const void *)status})
    if (!aligned(a, 4)) return MFD_ERR_INVALID_ARG;
  if (normalize != 0 && (normalize != 1 || !(eps >= 0.f) || !std::isfinite(eps))) return MFD_ERR_INVALID_ARG;
  if (state->Dk % 16 != 0 || state->Dk > 128 || state->Dv % 16 != 0 || state->Dv > 256 || state->Hv > 1024 ||
      state->Hv % Hk != 0)
    return MFD_ERR_UNSUPPORTED;
  if (!rows_ok(k, k_stride, Hk, state->Dk) || !rows_ok(v, v_stride, state->Hv, state->Dv)) return MFD_ERR_INVALID_ARG;
  if ((int64_t)n_req * N >= ((int64_t)1 << 31) - 1 || (int64_t)n_req * state->Hv * 8 >= ((int64_t)1 << 31) - 1)
    return MFD_ERR_UNSUPPORTED;
  *A = mfd::DeltaArgs{};
  A->k = static_cast<const uint16_t *>(k);
  A->v = static_cast<const uint16_t *>(v);
  A->k_stride = k_stride;
  A->v_stride = v_stride;
  A->dtype = dtype;
  A->n_req = n_req;
  A->N = N;
  A->Hk = Hk;
  A->Hv = state->Hv;
  A->Dk = state->Dk;
  A->Dv = state->Dv;
  A->g = g;
  A->beta = beta;
  A->normalize = normalize;
  A->eps = eps;
  A->n_nodes = n_nodes;
  A->s = state->s;
  A->n_slots = state->n_slots;
  A->src = src;
  A->dst = dst;
  A->status = status;
  return MFD_OK;
}

// The queries and outputs of the two forms that have them.
int delta_out(const void *q, int64_t q_stride, float scale, void *out, mfd::DeltaArgs *A) {
  if (!rows_ok(q, q_stride, A->Hk, A->Dk) || !out || !aligned(out, 16) || !std::isfinite(scale)) return MFD_ERR_INVALID_ARG;
  A->q = static_cast<const uint16_t *>(q);
  A->q_stride = q_stride;
  A->scale = scale;
  A->out = static_cast<uint16_t *>(out);
  return MFD_OK;
}

bool act_ok(int act) { return act == MFD_ACT_NONE || act == MFD_ACT_SIGMOID || act == MFD_ACT_SILU; }

}  // namespace

extern "C" {

int mfd_delta_rule(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                   int dtype, int n_req, int N, int Hk, const float *g, const float *beta, int normalize, float eps,
                   float scale, const int32_t *n_nodes, void *out, const mfd_delta_state *state, const int32_t *src,
                   const int32_t *dst, int32_t *status, mfd_stream_t stream) {
  mfd::DeltaArgs A;
  int rc = delta_args(k, k_stride, v, v_stride, dtype, n_req, N, Hk, g, beta, normalize, eps, n_nodes, state, src, dst, status, &A);
  if (rc != MFD_OK || (rc = delta_out(q, q_stride, scale, out, &A)) != MFD_OK) return rc;
  DeviceInfo d;
  if ((rc = current_device_info(&d)) != MFD_OK) return rc;
  if (!is_sm103(d)) return MFD_ERR_UNSUPPORTED;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(N >= mfd::DELTA_CHUNK_FROM ? mfd::launch_delta_chunk(A, cs) : mfd::launch_delta_rows(A, d.n_sm, cs));
}

int mfd_delta_tree(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                   int dtype, int n_req, int N, int Hk, const float *g, const float *beta, int normalize, float eps,
                   float scale, const int32_t *parent, const int32_t *n_nodes, void *out, const mfd_delta_state *state,
                   const int32_t *src, int32_t *status, mfd_stream_t stream) {
  mfd::DeltaArgs A;
  int rc = delta_args(k, k_stride, v, v_stride, dtype, n_req, N, Hk, g, beta, normalize, eps, n_nodes, state, src, nullptr, status, &A);
  if (rc != MFD_OK || (rc = delta_out(q, q_stride, scale, out, &A)) != MFD_OK) return rc;
  if (!parent || !aligned(parent, 4)) return MFD_ERR_INVALID_ARG;
  if (N > mfd::DELTA_MAX_NODES) return MFD_ERR_UNSUPPORTED;
  A.parent = parent;
  DeviceInfo d;
  if ((rc = current_device_info(&d)) != MFD_OK) return rc;
  if (!is_sm103(d)) return MFD_ERR_UNSUPPORTED;
  return cuda_status(mfd::launch_delta_tree(A, d.n_sm, reinterpret_cast<cudaStream_t>(stream)));
}

int mfd_delta_commit(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int dtype, int n_req, int N,
                     int Hk, const float *g, const float *beta, int normalize, float eps, int L,
                     const int32_t *accept_len, const int32_t *path_nodes, const int32_t *n_nodes,
                     const mfd_delta_state *state, const int32_t *src, const int32_t *dst, int32_t *status,
                     mfd_stream_t stream) {
  mfd::DeltaArgs A;
  int rc = delta_args(k, k_stride, v, v_stride, dtype, n_req, N, Hk, g, beta, normalize, eps, n_nodes, state, src, dst, status, &A);
  if (rc != MFD_OK) return rc;
  if (!accept_len || !path_nodes || !aligned(accept_len, 4) || !aligned(path_nodes, 4) || L < 1) return MFD_ERR_INVALID_ARG;
  if (L > 16) return MFD_ERR_UNSUPPORTED;
  A.accept_len = accept_len;
  A.path = path_nodes;
  A.L = L;
  DeviceInfo d;
  if ((rc = current_device_info(&d)) != MFD_OK) return rc;
  if (!is_sm103(d)) return MFD_ERR_UNSUPPORTED;
  return cuda_status(mfd::launch_delta_commit(A, d.n_sm, reinterpret_cast<cudaStream_t>(stream)));
}

int mfd_gated_norm(const void *x, int64_t x_stride, const void *gate, int64_t gate_stride, int dtype, int T, int heads,
                   int D, const void *w, float eps, int act, void *out, mfd_stream_t stream) {
  if (T < 1 || heads < 1 || D < 1 || !w || !aligned(w, 16) || !out || !aligned(out, 16)) return MFD_ERR_INVALID_ARG;
  if (dtype != MFD_BF16 && dtype != MFD_FP16) return MFD_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !act_ok(act)) return MFD_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 256 || heads > 1024 || (int64_t)T * heads >= ((int64_t)1 << 31) - 1) return MFD_ERR_UNSUPPORTED;
  if (!rows_ok(x, x_stride, heads, D) || !rows_ok(gate, gate_stride, heads, D)) return MFD_ERR_INVALID_ARG;
  const int rc = need_sm103();
  if (rc != MFD_OK) return rc;
  mfd::GatedNormArgs A;
  A.x = static_cast<const uint16_t *>(x);
  A.gate = static_cast<const uint16_t *>(gate);
  A.w = static_cast<const uint16_t *>(w);
  A.x_stride = x_stride;
  A.gate_stride = gate_stride;
  A.dtype = dtype;
  A.T = T;
  A.heads = heads;
  A.D = D;
  A.act = act;
  A.eps = eps;
  A.out = static_cast<uint16_t *>(out);
  return cuda_status(mfd::launch_gated_norm(A, reinterpret_cast<cudaStream_t>(stream)));
}

int mfd_residual_norm(const void *y, const void *residual, int dtype, int T, int H, const void *w_post,
                      const void *gate, int64_t gate_stride, int act, float scale, const void *w_pre, float eps,
                      void *residual_out, void *x_out, mfd_stream_t stream) {
  if (T < 1 || H < 1 || !y || !residual || !residual_out) return MFD_ERR_INVALID_ARG;
  if ((w_pre != nullptr) != (x_out != nullptr)) return MFD_ERR_INVALID_ARG;
  for (const void *a : {y, residual, w_post, gate, w_pre, (const void *)residual_out, (const void *)x_out})
    if (a && !aligned(a, 16)) return MFD_ERR_INVALID_ARG;
  if (dtype != MFD_BF16 && dtype != MFD_FP16) return MFD_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(scale) || !act_ok(act)) return MFD_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > 16384) return MFD_ERR_UNSUPPORTED;
  if (gate && gate_stride != 0 && (gate_stride < H || gate_stride % 8 != 0 || gate_stride >= ((int64_t)1 << 40)))
    return MFD_ERR_INVALID_ARG;
  if (residual_out == x_out) return MFD_ERR_INVALID_ARG;
  DeviceInfo d;
  const int rc = current_device_info(&d);
  if (rc != MFD_OK) return rc;
  if (!is_sm103(d)) return MFD_ERR_UNSUPPORTED;
  mfd::ResidualNormArgs A;
  A.y = static_cast<const uint16_t *>(y);
  A.residual = static_cast<const uint16_t *>(residual);
  A.w_post = static_cast<const uint16_t *>(w_post);
  A.gate = static_cast<const uint16_t *>(gate);
  A.w_pre = static_cast<const uint16_t *>(w_pre);
  A.gate_stride = gate_stride;
  A.dtype = dtype;
  A.T = T;
  A.H = H;
  A.act = act;
  A.scale = scale;
  A.eps = eps;
  A.residual_out = static_cast<uint16_t *>(residual_out);
  A.x_out = static_cast<uint16_t *>(x_out);
  return cuda_status(mfd::launch_residual_norm(A, d.n_sm, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
