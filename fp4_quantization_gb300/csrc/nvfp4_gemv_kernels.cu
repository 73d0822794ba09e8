// nvfp4_gemv_kernels.cu -- few rows times NVFP4 weights.
//
// out[r, n] = G_e * sum_k x[r / share, k] * s[n, k / 16] * c[n, k] for the
// expert e of row r, with E2M1 codes c, E4M3 scales s and the fp32 scale G_e.
#include "mxq_products.h"

#include "mxq_ptx.cuh"

namespace mxq {
namespace {

constexpr int WARPS = 8;
constexpr int ROWS = 4;        // rows of x that one pass over the weights serves
constexpr int LIST = 1024;     // row numbers scanned at a time

// Two E2M1 codes (one byte) as fp32.
__device__ __forceinline__ float2 e2m1x2_to_f32(uint32_t byte) {
  uint32_t h2;
  asm("{\n\t.reg .b8 b, z;\n\t"
      ".reg .b16 w;\n\t"
      "cvt.u16.u32 w, %1;\n\t"
      "mov.b16 {b, z}, w;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h2) : "r"(byte));
  return __half22float2(*reinterpret_cast<__half2*>(&h2));
}

__device__ __forceinline__ void store_out(const GemvArgs& a, int64_t row, int n, float v) {
  if (a.out_f32) {
    static_cast<float*>(a.out)[row * a.ldo + n] = v;
  } else {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(0.f), "f"(v));
    static_cast<uint16_t*>(a.out)[row * a.ldo + n] = static_cast<uint16_t>(d);
  }
}

// A warp an output column, an expert a grid row; lanes stride over K in
// 32-value pieces.
__global__ void __launch_bounds__(32 * WARPS) nvfp4_gemv_kernel(const GemvArgs a) {
  __shared__ int list[LIST];
  __shared__ int count;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int e = blockIdx.y;
  const int n = blockIdx.x * WARPS + warp;
  const float g = a.w_global[e];
  const uint8_t* q = a.w_q + (static_cast<int64_t>(e) * a.n + n) * (a.k / 2);
  const uint8_t* s = a.w_s + (static_cast<int64_t>(e) * a.n + n) * (a.k / 16);

  for (int from = 0; from < a.rows; from += LIST) {
    const int seen = min(LIST, a.rows - from);
    __syncthreads();
    if (tid == 0) count = 0;
    __syncthreads();
    // This expert's rows; expert 0 also clears the rows that have none.
    for (int i = tid; i < seen; i += 32 * WARPS) {
      const int id = a.experts ? a.experts[from + i] : 0;
      if (id == e) list[atomicAdd(&count, 1)] = from + i;
      if (e == 0 && (id < 0 || id >= a.num_experts))
        for (int j = 0; j < WARPS; ++j)
          if (blockIdx.x * WARPS + j < a.n) store_out(a, from + i, blockIdx.x * WARPS + j, 0.f);
    }
    __syncthreads();
    if (n >= a.n) continue;
    for (int r0 = 0; r0 < count; r0 += ROWS) {
      const uint16_t* x[ROWS];
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        x[i] = a.x + (list[min(r0 + i, count - 1)] / a.share) * a.ldx;
      float acc[ROWS] = {};
      for (int k = lane * 32; k < a.k; k += 1024) {
        const uint4 c4 = __ldg(reinterpret_cast<const uint4*>(q + k / 2));
        const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
        const uint32_t sc = __ldg(reinterpret_cast<const uint16_t*>(s + k / 16));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // The weight's value, with both scales, before x enters: x times a
          // code alone could leave fp32's range.
          const float d = e4m3_to_f32(sc >> (8 * h)) * g;
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const float2 v = e2m1x2_to_f32((c[2 * h + w] >> (8 * b)) & 0xFF);
              const int at = k + 16 * h + 8 * w + 2 * b;
#pragma unroll
              for (int i = 0; i < ROWS; ++i) {
                const uint32_t p = __ldg(reinterpret_cast<const uint32_t*>(x[i] + at));
                acc[i] += v.x * d * bf16_lo(p);
                acc[i] += v.y * d * bf16_hi(p);
              }
            }
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
#pragma unroll
        for (int m = 16; m > 0; m /= 2) acc[i] += __shfl_xor_sync(~0u, acc[i], m);
        if (lane == 0 && r0 + i < count) store_out(a, list[r0 + i], n, acc[i]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_nvfp4_gemv(const GemvArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const dim3 grid((a.n + WARPS - 1) / WARPS, a.experts ? a.num_experts : 1);
  nvfp4_gemv_kernel<<<grid, 32 * WARPS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mxq
