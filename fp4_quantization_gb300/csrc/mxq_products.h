// mxq_products.h -- launch arguments and launchers of the products on
// block-scaled operands, and the host helpers of mxq_api.cu that their entry
// points share.  Not installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "mxq.h"

namespace mxq {

constexpr int GROUPS_MAX = 512;       // experts of one grouped call
constexpr uint64_t PRODUCT_TIMEOUT_NS = 1000000000ull;   // 1 s per wait

// One grouped product: tiles of out = A B^T, where A's and B's rows are codes
// along the contraction axis.  Forward: A is [limit][depth], B is
// [groups][b_rows][depth], and group g owns A's (and out's) rows
// [offsets[g], offsets[g + 1]).  With few rows (GroupedPlan::few) the same with
// A and B exchanged: A is [groups][a_rows][depth], B is [limit][depth].  Weight
// gradient: A is [a_rows][limit], B is [b_rows][limit], and group g owns the
// contraction range [offsets[g], offsets[g + 1]) and the output matrix g.
struct GroupedArgs {
  const int32_t* offsets;   // [groups + 1], device
  int groups;
  int limit;                // M: no offset is above it
  int a_rows;               // wgrad, few: N
  int b_rows;               // forward: N; wgrad: K
  int depth;                // forward: K
  int split;                // GroupedPlan::split
  const uint8_t* a_s;       // E8M0 scales, s_ld bytes a row
  const uint8_t* b_s;
  int64_t s_ld;
  void* out;
  int64_t ldo;              // elements between output rows
  int out_f32;              // 1: fp32, 0: bf16
  int out_vec;              // output rows start on 16-byte boundaries
  uint32_t* dev_err;
  uint64_t timeout_ns;
};

struct GroupedMaps {
  CUtensorMap a;            // 3-D codes (depth, row, group), box 128 bytes x 128 rows x 1, 128-byte
                            // swizzle
  CUtensorMap b;            // the same, box 128 bytes x GroupedPlan::box_rows() x 1
  CUtensorMap out;          // 3-D output (column, row, group), box 128 bytes x 32 rows x 1, 128-byte
                            // swizzle; unset unless GroupedArgs::out_vec
};

// How a call's output is cut: tiles of 128 * ctas rows (a pair of CTAs works on
// one where ctas is 2) and `cols` columns.
struct GroupedPlan {
  int ctas;
  int cols;
  bool few;                // few rows a group: they are B, and the weight A
  int split;               // CTAs of a cluster that share a tile's contraction, or 1
  int64_t tiles;           // at most this many
  int grid;                // CTAs launched
  int box_rows() const { return cols / ctas; }   // rows of one copy of B
};

// The plan of mx_grouped_gemm, or of mx_grouped_wgrad, for sizes that are not
// empty.
GroupedPlan grouped_plan(int64_t M, int64_t N, int64_t K, int64_t groups, bool wgrad,
                         bool out_f32, int num_sms);
cudaError_t launch_grouped(const GroupedMaps& maps, const GroupedArgs& a, bool wgrad,
                           const GroupedPlan& plan, cudaStream_t stream);

constexpr int GEMV_EXPERTS_MAX = 4096;

struct GemvArgs {
  const uint16_t* x;        // bf16 [rows / share][ldx]
  int64_t ldx;
  int rows, n, k;
  const uint8_t* w_q;       // [experts][n][k / 2]
  const uint8_t* w_s;       // [experts][n][k / 16]
  const float* w_global;    // [experts]
  const int32_t* experts;   // [rows] or null
  int num_experts;
  int share;
  void* out;
  int64_t ldo;
  int out_f32;
  uint32_t* dev_err;
  uint64_t timeout_ns;
};

// How a call is cut: 16 * tiles output columns a CTA, K over clusters, at most
// `cap` rows of x at a time, by the kernel for up to `toks` (8 or 16).
struct GemvPlan {
  int toks;
  int tiles, cluster, cap;
  bool uneven;             // how much of K is staged follows each expert's rows
  int64_t items;           // experts that may have rows, times their blocks of columns
  int grid;                // CTAs launched
};

// The plan for `rows` output rows; experts is 0 for one weight and no ids.
GemvPlan gemv_plan(int64_t rows, int64_t n, int64_t k, int64_t experts, int num_sms);
cudaError_t launch_nvfp4_gemv(const GemvArgs& a, const GemvPlan& plan, cudaStream_t stream);

// Host helpers (mxq_api.cu).
// Allows `kernel` (a __global__ function) `bytes` of dynamic shared memory on the
// current device; asks the runtime once for each device (*done holds a bit for
// each), as the question takes longer than the rest of a launch's preparation.
cudaError_t allow_shared(const void* kernel, int bytes, std::atomic<uint64_t>* done);
mxq_status current_device(int* num_sms);
mxq_status encode_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base,
                      const cuuint64_t* dims, const cuuint64_t* strides_bytes,
                      const cuuint32_t* box,
                      CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_NONE);

}  // namespace mxq
