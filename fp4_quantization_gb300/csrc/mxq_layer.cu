// mxq_layer.cu -- the extern "C" entry points of the operators around the products
// (include/mxq.h): argument checks, tensor maps and dispatch.  Host code only; it
// allocates nothing and never synchronises.
#include <cmath>
#include <cstdint>

#include "mxq.h"
#include "mxq_internal.h"
#include "mxq_layer.h"
#include "mxq_products.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mxq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MXQ_OK : MXQ_ECUDA; }

constexpr int64_t kMost = int64_t(1) << 30;
constexpr int64_t kMostValues = int64_t(1) << 40;

constexpr uint32_t kDirections = MXQ_ROWWISE | MXQ_COLWISE;
constexpr uint32_t kScales = MXQ_SCALE_RCEIL | MXQ_SCALE_SWIZZLED;

mxq_status check_outputs(uint32_t flags, const uint8_t* q_row, const uint8_t* s_row,
                         const uint8_t* q_col, const uint8_t* s_col) {
  if ((flags & MXQ_ROWWISE) && (!q_row || !s_row)) return MXQ_EINVAL;
  if ((flags & MXQ_COLWISE) && (!q_col || !s_col)) return MXQ_EINVAL;
  if ((flags & MXQ_ROWWISE) && (!aligned(q_row, 16) || !aligned(s_row, 16))) return MXQ_EALIGN;
  if ((flags & MXQ_COLWISE) && (!aligned(q_col, 16) || !aligned(s_col, 16))) return MXQ_EALIGN;
  return MXQ_OK;
}

int direction_mode(uint32_t flags) {
  return ((flags & MXQ_ROWWISE) ? mxq::MX_ROW : 0) | ((flags & MXQ_COLWISE) ? mxq::MX_COL : 0);
}

// A bf16 matrix's pointer and stride, 16-byte rows.
bool rows_aligned(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

// Whether 32 bytes can be accessed at a time.
bool wide_rows(const void* p, int64_t ld) { return aligned(p, 32) && ld % 16 == 0; }

// The 8-bit checkpoint's codes [M][2N]: box 128 columns x a tile's rows, no swizzle.
mxq_status encode_saved_map(CUtensorMap* map, const uint8_t* q, int64_t M, int64_t N) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(2 * N), static_cast<cuuint64_t>(M)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(2 * N)};
  const cuuint32_t box[2] = {mxq::MX_TILE_K, static_cast<cuuint32_t>(mxq::saved_tile_rows())};
  return mxq::encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace

extern "C" {

mxq_status mx_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                      const void* weight, int64_t M, int64_t K, float eps, uint32_t flags, void* h,
                      int64_t ldh, float* rstd, void* y, int64_t ldy, uint8_t* q_row,
                      uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, uint32_t* dev_err,
                      mxq_stream_t stream) {
  if (flags & ~(kDirections | kScales | MXQ_OUT_BF16 | MXQ_IN_F32)) return MXQ_EINVAL;
  if (!(flags & (kDirections | MXQ_OUT_BF16))) return MXQ_EINVAL;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return MXQ_EINVAL;
  const bool col = (flags & MXQ_COLWISE) != 0, out = (flags & MXQ_OUT_BF16) != 0;
  if (M < 0 || K < 0 || M > kMost || K > mxq::NORM_K_MAX || M * K > kMostValues) return MXQ_ESHAPE;
  if (K % 32 || (col && M % 32)) return MXQ_ESHAPE;
  if (ldx < K || (residual && ldr < K) || (h && ldh < K) || (out && ldy < K)) return MXQ_ESHAPE;
  // Without a residual h would be x; with one the column pass reads it.
  if (!residual ? h != nullptr : (col && !h)) return MXQ_EINVAL;
  int sms = 0;
  mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (M == 0 || K == 0) return MXQ_OK;
  if (!x || !weight || !rstd || (out && !y)) return MXQ_EINVAL;
  if (!rows_aligned(x, ldx) || !aligned(weight, 16) || !aligned(rstd, 16)) return MXQ_EALIGN;
  if ((residual && !rows_aligned(residual, ldr)) || (h && !rows_aligned(h, ldh)) ||
      (out && !rows_aligned(y, ldy)))
    return MXQ_EALIGN;
  st = check_outputs(flags, q_row, s_row, q_col, s_col);
  if (st != MXQ_OK) return st;

  mxq::NormArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldh = ldh;
  a.ldy = ldy;
  a.weight = weight;
  a.weight_f32 = (flags & MXQ_IN_F32) != 0;
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.scale_ceil = (flags & MXQ_SCALE_RCEIL) != 0;
  a.scale_tiled = (flags & MXQ_SCALE_SWIZZLED) != 0;
  // Scale tiles are written whole: their padding rows are zeros.
  a.rows = a.scale_tiled && (flags & MXQ_ROWWISE) ? (a.M + 127) / 128 * 128 : a.M;
  a.eps = eps;
  a.inv_k = 1.0f / static_cast<float>(K);
  a.h = static_cast<uint16_t*>(h);
  a.rstd = rstd;
  if (out) a.y = static_cast<uint16_t*>(y);
  if (flags & MXQ_ROWWISE) {
    a.q_row = q_row;
    a.s_row = s_row;
  }
  a.wide = wide_rows(x, ldx) | wide_rows(residual, ldr) << 1 | wide_rows(h, ldh) << 2 |
           wide_rows(y, ldy) << 3;
  if (!col) return from_cuda(mxq::launch_norm_rows(a, sms, stream));

  CUtensorMap in, q;
  st = mxq::encode_bf16_map(&in, residual ? h : x, M, K, residual ? ldh : ldx, mxq::MX_TILE_K,
                            mxq::norm_tile_rows());
  if (st != MXQ_OK) return st;
  st = mxq::encode_mx_qcol_map(&q, M, K, q_col, mxq::norm_tile_rows());
  if (st != MXQ_OK) return st;
  return from_cuda(mxq::launch_norm_both(in, q, a, s_col, dev_err, mxq::LAYER_TIMEOUT_NS, sms, stream));
}

mxq_status mx_rmsnorm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh,
                               const float* rstd, const void* weight, const void* dh, int64_t lddh,
                               int64_t M, int64_t K, uint32_t flags, void* dx, int64_t lddx,
                               float* dweight, void* workspace, size_t workspace_bytes,
                               uint32_t* dev_err, mxq_stream_t stream) {
  if (flags & ~static_cast<uint32_t>(MXQ_IN_F32)) return MXQ_EINVAL;
  if (M < 0 || K < 0 || M > kMost || K > mxq::NORM_K_MAX || M * K > kMostValues) return MXQ_ESHAPE;
  if (K % 32) return MXQ_ESHAPE;
  if (lddy < K || ldh < K || lddx < K || (dh && lddh < K)) return MXQ_ESHAPE;
  if (!aligned(dweight, 16)) return MXQ_EALIGN;
  int sms = 0;
  mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (M == 0 || K == 0) {
    if (dweight && K > 0)
      return from_cuda(cudaMemsetAsync(dweight, 0, static_cast<size_t>(K) * sizeof(float), stream));
    return MXQ_OK;
  }
  if (!dy || !h || !rstd || !weight || !dx) return MXQ_EINVAL;
  if (!rows_aligned(dy, lddy) || !rows_aligned(h, ldh) || !rows_aligned(dx, lddx) ||
      (dh && !rows_aligned(dh, lddh)) || !aligned(weight, 16) || !aligned(rstd, 4))
    return MXQ_EALIGN;
  const int parts = mxq::norm_back_parts(M, K, sms);
  if (dweight) {
    if (!workspace || workspace_bytes < static_cast<size_t>(parts) * K * sizeof(float))
      return MXQ_EWORKSPACE;
    if (!aligned(workspace, 16)) return MXQ_EALIGN;
  }
  mxq::NormBackArgs a{};
  a.dy = static_cast<const uint16_t*>(dy);
  a.h = static_cast<const uint16_t*>(h);
  a.dh = static_cast<const uint16_t*>(dh);
  a.lddy = lddy;
  a.ldh = ldh;
  a.lddh = lddh;
  a.lddx = lddx;
  a.rstd = rstd;
  a.weight = weight;
  a.weight_f32 = (flags & MXQ_IN_F32) != 0;
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.inv_k = 1.0f / static_cast<float>(K);
  a.dx = static_cast<uint16_t*>(dx);
  a.parts = dweight ? static_cast<float*>(workspace) : nullptr;
  a.dev_err = dev_err;
  a.timeout_ns = mxq::LAYER_TIMEOUT_NS;
  return from_cuda(mxq::launch_norm_back(a, parts, dweight, stream));
}

mxq_status mx_quantize_gated_save(const void* x, int64_t M, int64_t N, int64_t ldx, uint32_t flags,
                                  uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                                  uint8_t* x_q, uint8_t* x_s, uint32_t* dev_err,
                                  mxq_stream_t stream) {
  if (flags & ~(kDirections | kScales | MXQ_ACT_GELU_TANH | MXQ_ACT_SILU)) return MXQ_EINVAL;
  if (!(flags & kDirections)) return MXQ_EINVAL;
  if ((flags & MXQ_ACT_GELU_TANH) && (flags & MXQ_ACT_SILU)) return MXQ_EINVAL;
  if (M < 0 || N < 0 || M > kMost || N > kMost / 2 || M * N > kMostValues) return MXQ_ESHAPE;
  if (ldx < 2 * N || M % 32 || N % 32) return MXQ_ESHAPE;
  int sms = 0;
  mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (M == 0 || N == 0) return MXQ_OK;
  if (!x || !x_q || !x_s) return MXQ_EINVAL;
  if (!rows_aligned(x, ldx) || !aligned(x_q, 16) || !aligned(x_s, 16)) return MXQ_EALIGN;
  st = check_outputs(flags, q_row, s_row, q_col, s_col);
  if (st != MXQ_OK) return st;
  mxq::SavedArgs a{};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.tiles_k = (a.N + mxq::MX_TILE_K - 1) / mxq::MX_TILE_K;
  a.ahead = mxq::saved_prefetch(sms);
  a.scale_ceil = (flags & MXQ_SCALE_RCEIL) != 0;
  a.scale_tiled = (flags & MXQ_SCALE_SWIZZLED) != 0;
  a.q_row = q_row;
  a.s_row = s_row;
  a.s_col = s_col;
  a.x_q = x_q;
  a.x_s = x_s;
  a.dev_err = dev_err;
  a.timeout_ns = mxq::LAYER_TIMEOUT_NS;
  mxq::SavedMaps maps{};
  st = mxq::encode_bf16_map(&maps.a, x, M, 2 * N, ldx, mxq::MX_TILE_K, mxq::saved_tile_rows());
  if (st != MXQ_OK) return st;
  if (flags & MXQ_COLWISE) {
    st = mxq::encode_mx_qcol_map(&maps.q_col, M, N, q_col, mxq::saved_tile_rows());
    if (st != MXQ_OK) return st;
  }
  return from_cuda(mxq::launch_gated_save(maps, a, direction_mode(flags),
                                          (flags & MXQ_ACT_GELU_TANH) != 0, stream));
}

mxq_status mx_quantize_dgated_saved(const void* grad, int64_t ldg, const uint8_t* x_q,
                                    const uint8_t* x_s, int64_t M, int64_t N, uint32_t flags,
                                    uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                                    uint32_t* dev_err, mxq_stream_t stream) {
  if (flags & ~(kDirections | kScales | MXQ_ACT_GELU_TANH | MXQ_ACT_SILU)) return MXQ_EINVAL;
  if (!(flags & kDirections)) return MXQ_EINVAL;
  if ((flags & MXQ_ACT_GELU_TANH) && (flags & MXQ_ACT_SILU)) return MXQ_EINVAL;
  if (M < 0 || N < 0 || M > kMost || N > kMost / 2 || M * N > kMostValues) return MXQ_ESHAPE;
  if (ldg < N || M % 32 || N % 32) return MXQ_ESHAPE;
  // Both halves' scale tiles have to start on a tile.
  if ((flags & MXQ_SCALE_SWIZZLED) && N % 128) return MXQ_ESHAPE;
  int sms = 0;
  mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (M == 0 || N == 0) return MXQ_OK;
  if (!grad || !x_q || !x_s) return MXQ_EINVAL;
  if (!rows_aligned(grad, ldg) || !aligned(x_q, 16) || !aligned(x_s, 16)) return MXQ_EALIGN;
  st = check_outputs(flags, q_row, s_row, q_col, s_col);
  if (st != MXQ_OK) return st;
  mxq::SavedArgs a{};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.tiles_k = (a.N + mxq::MX_TILE_K - 1) / mxq::MX_TILE_K;
  a.scale_ceil = (flags & MXQ_SCALE_RCEIL) != 0;
  a.scale_tiled = (flags & MXQ_SCALE_SWIZZLED) != 0;
  a.q_row = q_row;
  a.s_row = s_row;
  a.s_col = s_col;
  a.saved_s = x_s;
  a.dev_err = dev_err;
  a.timeout_ns = mxq::LAYER_TIMEOUT_NS;
  mxq::SavedMaps maps{};
  st = mxq::encode_bf16_map(&maps.a, grad, M, N, ldg, mxq::MX_TILE_K, mxq::saved_tile_rows());
  if (st != MXQ_OK) return st;
  st = encode_saved_map(&maps.b, x_q, M, N);
  if (st != MXQ_OK) return st;
  if (flags & MXQ_COLWISE) {
    st = mxq::encode_mx_qcol_map(&maps.q_col, M, N, q_col, mxq::saved_tile_rows());
    if (st != MXQ_OK) return st;
    st = mxq::encode_mx_qcol_map(&maps.q_col2, M, N, q_col + N * M, mxq::saved_tile_rows());
    if (st != MXQ_OK) return st;
  }
  return from_cuda(mxq::launch_dgated_saved(maps, a, direction_mode(flags),
                                            (flags & MXQ_ACT_GELU_TANH) != 0, stream));
}

mxq_status moe_route(const void* logits, int64_t ldl, const float* bias, int64_t T, int64_t E,
                     int64_t k, int64_t groups, int64_t kept, float scale, uint32_t flags,
                     int32_t* experts, float* weights, mxq_stream_t stream) {
  if (flags & ~static_cast<uint32_t>(MXQ_IN_F32 | MXQ_ROUTE_SIGMOID | MXQ_ROUTE_RENORM | MXQ_ROUTE_GROUP_MAX))
    return MXQ_EINVAL;
  if (!std::isfinite(scale)) return MXQ_EINVAL;
  if (T < 0 || T > kMost || E < 1 || E > mxq::ROUTE_EXPERTS_MAX || ldl < E || ldl > kMost) return MXQ_ESHAPE;
  if (groups < 1 || groups > mxq::ROUTE_GROUPS_MAX || E % groups || kept < 1 || kept > groups)
    return MXQ_ESHAPE;
  if (k < 1 || k > mxq::ROUTE_SLOTS_MAX || k > E / groups * kept) return MXQ_ESHAPE;
  int sms = 0;
  const mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (T == 0) return MXQ_OK;
  if (!logits || !experts || !weights) return MXQ_EINVAL;
  if (!aligned(logits, flags & MXQ_IN_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(experts, 4) ||
      !aligned(weights, 4))
    return MXQ_EALIGN;
  mxq::RouteArgs a{};
  a.logits = logits;
  a.ldl = ldl;
  a.bias = bias;
  a.tokens = static_cast<int>(T);
  a.experts = static_cast<int>(E);
  a.slots = static_cast<int>(k);
  a.groups = static_cast<int>(groups);
  a.kept = static_cast<int>(kept);
  a.scale = scale;
  a.flags = flags;
  a.ids = experts;
  a.weights = weights;
  return from_cuda(mxq::launch_route(a, stream));
}

mxq_status moe_route_backward(const float* dweights, const void* logits, int64_t ldl,
                              const int32_t* experts, int64_t T, int64_t E, int64_t k, float scale,
                              uint32_t flags, void* dlogits, int64_t ldd, mxq_stream_t stream) {
  if (flags & ~static_cast<uint32_t>(MXQ_IN_F32 | MXQ_ROUTE_SIGMOID | MXQ_ROUTE_RENORM))
    return MXQ_EINVAL;
  if (!std::isfinite(scale)) return MXQ_EINVAL;
  if (T < 0 || T > kMost || E < 1 || E > mxq::ROUTE_EXPERTS_MAX || ldl < E || ldd < E ||
      ldl > kMost || ldd > kMost)
    return MXQ_ESHAPE;
  if (k < 1 || k > mxq::ROUTE_SLOTS_MAX) return MXQ_ESHAPE;
  int sms = 0;
  const mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (T == 0) return MXQ_OK;
  if (!dweights || !logits || !experts || !dlogits) return MXQ_EINVAL;
  const int size = flags & MXQ_IN_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(experts, 4) ||
      !aligned(dweights, 4))
    return MXQ_EALIGN;
  mxq::RouteBackArgs a{};
  a.dweights = dweights;
  a.logits = logits;
  a.ldl = ldl;
  a.ids = experts;
  a.tokens = static_cast<int>(T);
  a.experts = static_cast<int>(E);
  a.slots = static_cast<int>(k);
  a.scale = scale;
  a.flags = flags;
  a.dlogits = dlogits;
  a.ldd = ldd;
  return from_cuda(mxq::launch_route_back(a, stream));
}

mxq_status moe_sort(const int32_t* experts, int64_t n, int64_t E, int64_t align, int32_t* rows,
                    int32_t* offsets, int32_t* sizes, int32_t* source, int64_t source_rows,
                    mxq_stream_t stream) {
  if (n < 0 || n > kMost || E < 1 || E > mxq::ROUTE_EXPERTS_MAX || align < 1 || align > 65536)
    return MXQ_ESHAPE;
  // Every row that the pairs and their padding can take, which has to fit int32.
  const int64_t most = n + (n < E ? n : E) * (align - 1);
  if (most > INT32_MAX || source_rows < 0 || source_rows > INT32_MAX) return MXQ_ESHAPE;
  if (source && source_rows < most) return MXQ_ESHAPE;
  int sms = 0;
  const mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (!offsets || (n > 0 && (!experts || !rows))) return MXQ_EINVAL;
  if (!aligned(experts, 4) || !aligned(rows, 4) || !aligned(offsets, 4) || !aligned(sizes, 4) ||
      !aligned(source, 4))
    return MXQ_EALIGN;
  mxq::SortArgs a{};
  a.ids = experts;
  a.n = n;
  a.experts = static_cast<int>(E);
  a.align = static_cast<int>(align);
  a.rows_max = source_rows;
  a.rows = rows;
  a.offsets = offsets;
  a.sizes = sizes;
  a.source = source;
  return from_cuda(mxq::launch_sort(a, stream));
}

}  // extern "C"
