// delta.h -- the recurrent layers' calls as kernels see them: the gated delta
// rule over rows, trees and accepted paths (delta_rows.cu,
// delta_chunk.cu, delta_tree.cu), and the norms with
// gates (norms.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mfd.h"

namespace mfd {

// What every form of the rule gets.  States are fp32 [n_slots][Hv][Dk][Dv].
struct DeltaArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  int dtype, n_req, N, Hk, Hv, Dk, Dv;
  const float *g, *beta;  // [n_req][N][Hv]
  int normalize;
  float eps, scale;
  const int32_t *n_nodes;
  float *s;
  int n_slots;
  const int32_t *src, *dst;
  uint16_t *out;  // [n_req][N][Hv][Dv]
  int32_t *status;
  const int32_t *parent;                 // tree: [n_req][N]
  const int32_t *accept_len, *path;      // commit: [n_req], [n_req][L + 1]
  int L;
};

constexpr int DELTA_MAX_DEPTH = 16;   // of a tree's nodes, the root's being 0
constexpr int DELTA_MAX_NODES = 513;

// Rows from which the rule goes by chunks: what the row form has shared memory for.
// 17 rows of 32 heads there and 18 here take 13.5 and 15.9 us for one request, 24 and 33
// for 8, 159 and 236 for 64; a row more costs the row form 0.6, 1.1 and 8 us.
constexpr int DELTA_CHUNK_FROM = 18;
cudaError_t launch_delta_rows(const DeltaArgs &A, int n_sm, cudaStream_t stream);
cudaError_t launch_delta_chunk(const DeltaArgs &A, cudaStream_t stream);
cudaError_t launch_delta_commit(const DeltaArgs &A, int n_sm, cudaStream_t stream);
cudaError_t launch_delta_tree(const DeltaArgs &A, int n_sm, cudaStream_t stream);

struct GatedNormArgs {
  const uint16_t *x, *gate, *w;
  int64_t x_stride, gate_stride;  // elements between tokens
  int dtype, T, heads, D, act;
  float eps;
  uint16_t *out;
};
cudaError_t launch_gated_norm(const GatedNormArgs &A, cudaStream_t stream);

struct ResidualNormArgs {
  const uint16_t *y, *residual, *w_post, *gate, *w_pre;
  int64_t gate_stride;  // 0: one row for all tokens
  int dtype, T, H, act;
  float scale, eps;
  uint16_t *residual_out, *x_out;
};
cudaError_t launch_residual_norm(const ResidualNormArgs &A, int n_sm, cudaStream_t stream);

}  // namespace mfd
