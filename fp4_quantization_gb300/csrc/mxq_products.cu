// mxq_products.cu -- the extern "C" entry points of the products on
// block-scaled operands (include/mxq.h): argument checks, tensor maps and
// dispatch.  Host code only; it allocates nothing and never synchronises.
#include <cstdint>

#include "mxq.h"
#include "mxq_products.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mxq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MXQ_OK : MXQ_ECUDA; }

constexpr int64_t kMost = int64_t(1) << 30;

// E4M3 codes [groups][rows][depth] (depth contiguous): box of one swizzle row
// of 128 codes x box_rows rows.
mxq_status encode_codes(CUtensorMap* map, const uint8_t* q, int64_t groups, int64_t rows,
                        int64_t depth, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(depth), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(groups)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(depth),
                                 static_cast<cuuint64_t>(depth * rows)};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows), 1};
  return mxq::encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, q, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

// Sets the output fields after checking them: [groups][rows][cols], ldo
// elements between rows.
mxq_status set_output(mxq::GroupedArgs* a, CUtensorMap* map, void* out, int64_t groups,
                      int64_t rows, int64_t cols, int64_t ldo, uint32_t flags) {
  const int size = (flags & MXQ_OUT_F32) ? 4 : 2;
  if (!aligned(out, size)) return MXQ_EALIGN;
  a->out = out;
  a->ldo = ldo;
  a->out_f32 = size == 4;
  a->out_vec = aligned(out, 16) && (ldo * size) % 16 == 0;
  if (!a->out_vec) return MXQ_OK;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(groups)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ldo * size),
                                 static_cast<cuuint64_t>(ldo * size * rows)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), 32, 1};
  return mxq::encode_map(map,
                         size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         3, out, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

extern "C" {

mxq_status mx_grouped_gemm(const uint8_t* x_q, const uint8_t* x_s, const uint8_t* w_q,
                           const uint8_t* w_s, const int32_t* offsets, int64_t M, int64_t N,
                           int64_t K, int64_t E, uint32_t flags, void* out, int64_t ldo,
                           uint32_t* dev_err, mxq_stream_t stream) {
  if (flags & ~static_cast<uint32_t>(MXQ_OUT_F32)) return MXQ_EINVAL;
  if (M < 0 || N < 0 || K < 0 || E < 0 || ldo < N) return MXQ_ESHAPE;
  if (K % 32) return MXQ_ESHAPE;
  if (M > kMost || N > kMost || K > kMost || E > mxq::GROUPS_MAX) return MXQ_ESHAPE;
  if ((M / 128 + E) * (N / 128 + 1) > kMost) return MXQ_ESHAPE;
  int sms = 0;
  mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (M == 0 || N == 0 || E == 0) return MXQ_OK;
  if (!offsets || !out) return MXQ_EINVAL;
  if (K > 0 && (!x_q || !x_s || !w_q || !w_s)) return MXQ_EINVAL;
  if (!aligned(x_q, 16) || !aligned(x_s, 16) || !aligned(w_q, 16) || !aligned(w_s, 16) ||
      !aligned(offsets, 4))
    return MXQ_EALIGN;
  mxq::GroupedArgs a{};
  mxq::GroupedMaps maps{};
  st = set_output(&a, &maps.out, out, 1, M, N, ldo, flags);
  if (st != MXQ_OK) return st;
  a.offsets = offsets;
  a.groups = static_cast<int>(E);
  a.limit = static_cast<int>(M);
  a.depth = static_cast<int>(K);
  a.s_ld = K / 32;
  a.dev_err = dev_err;
  a.timeout_ns = mxq::PRODUCT_TIMEOUT_NS;
  const mxq::GroupedPlan plan = mxq::grouped_plan(M, N, K, E, false, a.out_f32, sms);
  a.split = plan.split;
  (plan.few ? a.a_rows : a.b_rows) = static_cast<int>(N);
  a.a_s = plan.few ? w_s : x_s;
  a.b_s = plan.few ? x_s : w_s;
  if (K > 0) {
    st = encode_codes(plan.few ? &maps.b : &maps.a, x_q, 1, M, K,
                      plan.few ? plan.box_rows() : 128);
    if (st != MXQ_OK) return st;
    st = encode_codes(plan.few ? &maps.a : &maps.b, w_q, E, N, K,
                      plan.few ? 128 : plan.box_rows());
    if (st != MXQ_OK) return st;
  }
  return from_cuda(mxq::launch_grouped(maps, a, false, plan, stream));
}

mxq_status mx_grouped_wgrad(const uint8_t* g_q, const uint8_t* g_s, const uint8_t* x_q,
                            const uint8_t* x_s, const int32_t* offsets, int64_t M, int64_t N,
                            int64_t K, int64_t E, uint32_t flags, void* dw, uint32_t* dev_err,
                            mxq_stream_t stream) {
  if (flags & ~static_cast<uint32_t>(MXQ_OUT_F32)) return MXQ_EINVAL;
  if (M < 0 || N < 0 || K < 0 || E < 0) return MXQ_ESHAPE;
  if (M % 32) return MXQ_ESHAPE;
  if (M > kMost || N > kMost || K > kMost || E > mxq::GROUPS_MAX) return MXQ_ESHAPE;
  if ((N / 128 + 1) * E > kMost || (N / 128 + 1) * E * (K / 128 + 1) > kMost) return MXQ_ESHAPE;
  int sms = 0;
  mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (N == 0 || K == 0 || E == 0) return MXQ_OK;
  if (!offsets || !dw) return MXQ_EINVAL;
  if (M > 0 && (!g_q || !g_s || !x_q || !x_s)) return MXQ_EINVAL;
  if (!aligned(g_q, 16) || !aligned(g_s, 16) || !aligned(x_q, 16) || !aligned(x_s, 16) ||
      !aligned(offsets, 4))
    return MXQ_EALIGN;
  mxq::GroupedArgs a{};
  mxq::GroupedMaps maps{};
  st = set_output(&a, &maps.out, dw, E, N, K, K, flags);
  if (st != MXQ_OK) return st;
  a.offsets = offsets;
  a.groups = static_cast<int>(E);
  a.limit = static_cast<int>(M);
  a.a_rows = static_cast<int>(N);
  a.b_rows = static_cast<int>(K);
  a.a_s = g_s;
  a.b_s = x_s;
  a.s_ld = M / 32;
  a.dev_err = dev_err;
  a.timeout_ns = mxq::PRODUCT_TIMEOUT_NS;
  const mxq::GroupedPlan plan = mxq::grouped_plan(M, N, K, E, true, a.out_f32, sms);
  a.split = plan.split;
  if (M > 0) {
    st = encode_codes(&maps.a, g_q, 1, N, M, 128);
    if (st != MXQ_OK) return st;
    st = encode_codes(&maps.b, x_q, 1, K, M, plan.box_rows());
    if (st != MXQ_OK) return st;
  }
  return from_cuda(mxq::launch_grouped(maps, a, true, plan, stream));
}

mxq_status nvfp4_gemv(const void* x, int64_t ldx, const uint8_t* w_q, const uint8_t* w_s,
                      const float* w_global, const int32_t* experts, int64_t T, int64_t share,
                      int64_t N, int64_t K, int64_t E, uint32_t flags, void* out, int64_t ldo,
                      uint32_t* dev_err, mxq_stream_t stream) {
  if (flags & ~static_cast<uint32_t>(MXQ_OUT_F32)) return MXQ_EINVAL;
  if (T < 0 || N < 0 || K < 0 || E < 0 || share < 1 || ldx < K || ldo < N) return MXQ_ESHAPE;
  if (!experts && (share != 1 || E != 1)) return MXQ_ESHAPE;
  if (K % 32) return MXQ_ESHAPE;
  if (T > kMost || share > kMost || T * share > kMost || N > kMost || K > kMost ||
      E > mxq::GEMV_EXPERTS_MAX || E * (N + 16) > kMost)
    return MXQ_ESHAPE;
  int sms = 0;
  const mxq_status st = mxq::current_device(&sms);
  if (st != MXQ_OK) return st;
  if (T == 0 || N == 0) return MXQ_OK;
  if (!out || (E > 0 && !w_global) || (K > 0 && (!x || (E > 0 && (!w_q || !w_s)))))
    return MXQ_EINVAL;
  const int size = (flags & MXQ_OUT_F32) ? 4 : 2;
  if (!aligned(x, 16) || (ldx % 8) || !aligned(w_q, 16) || !aligned(w_s, 16) ||
      !aligned(w_global, 4) || !aligned(experts, 4) || !aligned(out, size))
    return MXQ_EALIGN;
  if (E == 0)
    return from_cuda(cudaMemset2DAsync(out, ldo * size, 0, N * size, T * share, stream));
  mxq::GemvArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.rows = static_cast<int>(T * share);
  a.n = static_cast<int>(N);
  a.k = static_cast<int>(K);
  a.w_q = w_q;
  a.w_s = w_s;
  a.w_global = w_global;
  a.experts = experts;
  a.num_experts = static_cast<int>(E);
  a.share = static_cast<int>(share);
  a.out = out;
  a.ldo = ldo;
  a.out_f32 = size == 4;
  a.dev_err = dev_err;
  a.timeout_ns = mxq::PRODUCT_TIMEOUT_NS;
  const mxq::GemvPlan plan = mxq::gemv_plan(a.rows, N, K, experts ? E : 0, sms);
  return from_cuda(mxq::launch_nvfp4_gemv(a, plan, stream));
}

mxq_status mxq_product_plan(int op, int64_t M, int64_t N, int64_t K, int64_t E, uint32_t flags,
                            int num_sms, int32_t* plan) {
  if (!plan || num_sms < 1 || (flags & ~static_cast<uint32_t>(MXQ_OUT_F32))) return MXQ_EINVAL;
  // Without rows a gradient is zeros, and without depth a product.
  const bool wgrad = op == MXQ_OP_GROUPED_WGRAD;
  if (M < (wgrad ? 0 : 1) || N < 1 || K < (wgrad ? 1 : 0) || M % (wgrad ? 32 : 1) ||
      K % (wgrad ? 1 : 32) || M > kMost || N > kMost || K > kMost)
    return MXQ_ESHAPE;
  if (wgrad || op == MXQ_OP_GROUPED_GEMM) {
    if (E < 1 || E > mxq::GROUPS_MAX) return MXQ_ESHAPE;
    const mxq::GroupedPlan p =
        mxq::grouped_plan(M, N, K, E, wgrad, (flags & MXQ_OUT_F32) != 0, num_sms);
    plan[0] = p.ctas;
    plan[1] = p.cols;
    plan[2] = p.few;
    plan[3] = p.split;
    plan[4] = p.tiles > INT32_MAX ? INT32_MAX : static_cast<int32_t>(p.tiles);
    plan[5] = p.grid;
    plan[6] = 0;
    return MXQ_OK;
  }
  if (op != MXQ_OP_NVFP4_GEMV) return MXQ_EINVAL;
  if (E < 0 || E > mxq::GEMV_EXPERTS_MAX) return MXQ_ESHAPE;
  const mxq::GemvPlan p = mxq::gemv_plan(M, N, K, E, num_sms);
  plan[0] = p.toks;
  plan[1] = p.tiles;
  plan[2] = p.cluster;
  plan[3] = p.cap;
  plan[4] = p.items > INT32_MAX ? INT32_MAX : static_cast<int32_t>(p.items);
  plan[5] = p.grid;
  plan[6] = p.uneven;
  return MXQ_OK;
}

}  // extern "C"
