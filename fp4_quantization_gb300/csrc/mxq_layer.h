// mxq_layer.h -- launch arguments and launchers of the operators around the
// products of a feed-forward block: RMSNorm, expert routing and sorting, and the
// gated activation with an 8-bit checkpoint.  Not installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "mxq.h"

namespace mxq {

constexpr uint64_t LAYER_TIMEOUT_NS = 1000000000ull;   // 1 s per wait

// ---- RMSNorm ----------------------------------------------------------------

constexpr int64_t NORM_K_MAX = 32768;   // 1024 threads hold 2 granules of 16 values each

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;   // or NULL
  int64_t ldx, ldr, ldh, ldy;
  const void* weight;         // bf16, or fp32 with weight_f32
  int weight_f32;
  int wide;                   // bits: rows of x, residual, h, y start on 32 bytes
  int M, K;
  int rows;                   // M, or M rounded up to 128 where scale tiles are padded
  float eps, inv_k;
  int scale_ceil, scale_tiled;
  uint16_t* h;                // or NULL
  float* rstd;
  uint16_t* y;                // or NULL
  uint8_t* q_row;             // or NULL
  uint8_t* s_row;
};

struct NormBackArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const uint16_t* dh;         // or NULL
  int64_t lddy, ldh, lddh, lddx;
  const float* rstd;
  const void* weight;
  int weight_f32;
  int M, K;
  float inv_k;
  uint16_t* dx;
  float* parts;               // [grid][K] column sums, or NULL
  uint32_t* dev_err;
  uint64_t timeout_ns;
};

cudaError_t launch_norm_rows(const NormArgs& a, int num_sms, cudaStream_t stream);
// The row pass and the column pass, with the maps of h (x without a residual) and of
// the colwise codes in boxes of norm_tile_rows() rows.
int norm_tile_rows();
cudaError_t launch_norm_both(const CUtensorMap& h, const CUtensorMap& q_col, const NormArgs& a,
                             uint8_t* s_col, uint32_t* dev_err, uint64_t timeout_ns, int num_sms,
                             cudaStream_t stream);
// CTAs of the backward pass, each of which leaves one row of column sums.
int norm_back_parts(int64_t M, int64_t K, int num_sms);
cudaError_t launch_norm_back(const NormBackArgs& a, int parts, float* dweight, cudaStream_t stream);

// ---- the gated activation with an 8-bit checkpoint -----------------------------

struct SavedArgs {
  int M, N;
  int tiles_k;                // 128-column tiles over N
  int ahead;                  // forward: tiles from one to that which it prefetches
  int scale_ceil, scale_tiled;
  uint8_t* q_row;
  uint8_t* s_row;
  uint8_t* s_col;
  uint8_t* x_q;               // forward: the checkpoint that is written
  uint8_t* x_s;
  const uint8_t* saved_s;     // backward: the checkpoint's scales
  uint32_t* dev_err;
  uint64_t timeout_ns;
};

struct SavedMaps {
  CUtensorMap a;              // forward: x, bf16; backward: grad, bf16
  CUtensorMap b;              // backward: the checkpoint's codes
  CUtensorMap q_col;          // colwise codes; backward: those of d gate
  CUtensorMap q_col2;         // backward: those of d up
};

// Rows of a tile, and how many tiles ahead the forward pass prefetches.
int saved_tile_rows();
int saved_prefetch(int num_sms);
cudaError_t launch_gated_save(const SavedMaps& maps, const SavedArgs& a, int mode, bool gelu,
                              cudaStream_t stream);
cudaError_t launch_dgated_saved(const SavedMaps& maps, const SavedArgs& a, int mode, bool gelu,
                                cudaStream_t stream);

// ---- routing and sorting ---------------------------------------------------------

constexpr int ROUTE_EXPERTS_MAX = 512;
constexpr int ROUTE_SLOTS_MAX = 32;     // one lane a slot
constexpr int ROUTE_GROUPS_MAX = 32;    // one lane a group

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  const float* bias;          // or NULL
  int tokens, experts, slots;
  int groups, kept;
  float scale;
  uint32_t flags;
  int32_t* ids;
  float* weights;
};

struct RouteBackArgs {
  const float* dweights;
  const void* logits;
  int64_t ldl;
  const int32_t* ids;
  int tokens, experts, slots;
  float scale;
  uint32_t flags;
  void* dlogits;
  int64_t ldd;
};

struct SortArgs {
  const int32_t* ids;
  int64_t n;
  int experts;
  int align;
  int64_t rows_max;           // entries of source
  int32_t* rows;
  int32_t* offsets;
  int32_t* sizes;             // or NULL
  int32_t* source;            // or NULL
};

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_route_back(const RouteBackArgs& a, cudaStream_t stream);
cudaError_t launch_sort(const SortArgs& a, cudaStream_t stream);

}  // namespace mxq
