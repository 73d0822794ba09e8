// mx_saved_kernels.cu -- the gated activation with an 8-bit checkpoint of its
// input, and the backward pass that reads the checkpoint.
//
// Forward: y = act(gate) * up of x = [gate | up] as MXFP8 along its rows and/or
// columns, and x itself as MXFP8 along its rows (blocks of 32 columns never reach
// from gate into up, as N % 32 == 0).  Backward: with x decoded from those codes
// and scales, d gate = grad * up * act'(gate) and d up = grad * act(gate).
//
// One CTA per 64 x 128 tile of y, taken in address order; its operands arrive by
// tensor copies (32 KiB: gate and up in bf16, or grad in bf16 and both in codes) and
// its results leave as mx_tile.cuh says.  8.2 bytes for each value of y, both ways out:
// 8192 x 14336 takes 147 us forward (0.96 of the copy rate, measured; 128-row tiles of
// 256 threads 190 us) and 169 us backward (0.84; 199 us), where the instructions of two
// outputs share the time with the traffic (rowwise alone: 1.04 and 0.89).

#include "mx_elements.cuh"
#include "mx_tile.cuh"
#include "mxq_internal.h"
#include "mxq_layer.h"
#include "mxq_products.h"
#include "mxq_ptx.cuh"

namespace mxq {
namespace {

// Rows a lane (mx_tile.cuh), four CTAs an SM each.  8192 x 14336, both ways out,
// measured on GB300 before the prefetch below: forward 153 us with 4 rows (32 warps an SM, 64 registers)
// and 165 us with 8 (three CTAs: 128 registers spill); backward, which issues twice the
// instructions a value, 180 us with 4 and 170 us with 8 (169 us since).
constexpr int SAVE_LR = 4, BACK_LR = 8;
constexpr int CTAS = 4;      // an SM
// Forward, a CTA has the operands of the tile half a wave on brought into L2 (CTAS / 2 an
// SM; with a whole wave 152 us, with two 192, without 156): its successor waits for L2
// instead of memory.  The backward pass waits for instructions: 168.4 us with, 168.7
// without.
constexpr int BF16_PITCH = MX_TILE_K * 2;
constexpr int BF16_TILE = TILE_ROWS * BF16_PITCH;
constexpr int CODE_TILE = TILE_ROWS * MX_TILE_K;

__device__ __forceinline__ float2 pair_of(uint32_t v) { return make_float2(bf16_lo(v), bf16_hi(v)); }

template <bool GELU>
__device__ __forceinline__ float2 gate_pair(float2 gate, float2 up) {
  return mul_f32x2(GELU ? gelu_tanh_pair(gate) : silu_pair(gate), up);
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// Rowwise MXFP8 of the lane's 4 x 8 bf16 values v: codes to q (row pitch `pitch`),
// scale bytes to [row][4] at `scales`.
__device__ __forceinline__ void save_block(const uint32_t (&v)[SAVE_LR][4], uint8_t* q,
                                           int64_t pitch, bool ok, uint32_t scales, int rl, int c,
                                           uint32_t ceil_bf16) {
  uint32_t rc[2];
#pragma unroll
  for (int i = 0; i < SAVE_LR; i += 2) {
    uint32_t t[2];
#pragma unroll
    for (int d = 0; d < 2; ++d)
      t[d] = absmax_bf16x2(absmax_bf16x2(v[i + d][0], v[i + d][1]),
                           absmax_bf16x2(v[i + d][2], v[i + d][3]));
    uint32_t e = bf16_scale_exponents(
        absmax_bf16x2(prmt(t[0], t[1], 0x5410), prmt(t[0], t[1], 0x7632)), ceil_bf16);
    e = vmax_u16x2(e, __shfl_xor_sync(0xFFFFFFFFu, e, 1));
    e = vmax_u16x2(e, __shfl_xor_sync(0xFFFFFFFFu, e, 2));
    rc[i / 2] = e8m0_pair(e);
  }
#pragma unroll
  for (int i = 0; i < SAVE_LR; ++i) {
    const float inv = i & 1 ? inv_scale_hi(rc[i >> 1]) : inv_scale_lo(rc[i >> 1]);
    uint32_t w[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 z = mul_f32x2(pair_of(v[i][p]), f2(inv));
      w[p] = cvt_e4m3x2(z.x, z.y);
    }
    if (ok) stg64_cs(q + i * pitch, w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  }
  sts8(scales + (rl + (c & 3)) * 4 + (c >> 2), half16(c & 2 ? rc[1] : rc[0], c & 1) & 0xFFu);
}

// The colwise staging takes the place of the gate's tile, which every warp has
// read by the first barrier of quantize_tile.
struct GatedSaveShared {
  static constexpr int UP = BF16_TILE;
  static constexpr int SCALES = 2 * BF16_TILE;
  static constexpr int SAVED = SCALES + Tile<SAVE_LR>::SCALES_BYTES;   // [2][rows][4]
  static constexpr int DYNAMIC = SAVED + 8 * TILE_ROWS + 1024;        // + alignment pad
};

template <int MODE, bool GELU>
__global__ void __launch_bounds__(Tile<SAVE_LR>::THREADS, CTAS)
mx_gated_save_kernel(const __grid_constant__ CUtensorMap tmap_x,
                     const __grid_constant__ CUtensorMap tmap_qcol, const SavedArgs a) {
  using L = GatedSaveShared;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full;
  const uint32_t sbase = smem_addr(align_up_shared<1024>(smem_raw));
  const uint32_t bar = smem_addr(&full);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = lane >> 4, c = lane & 15;
  const int band = static_cast<int>(blockIdx.x) / a.tiles_k;
  const int tk = static_cast<int>(blockIdx.x) - band * a.tiles_k;
  const int row0 = band * TILE_ROWS, col0 = tk * MX_TILE_K;
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
    mbar_arrive_expect_tx(bar, 2 * BF16_TILE);
    tma_load_2d(sbase, &tmap_x, col0, row0, bar);
    tma_load_2d(sbase + L::UP, &tmap_x, a.N + col0, row0, bar);
    const int tile = static_cast<int>(blockIdx.x) + a.ahead;
    if (tile < static_cast<int>(gridDim.x)) {
      const int x = tile % a.tiles_k * MX_TILE_K, y = tile / a.tiles_k * TILE_ROWS;
      tma_prefetch_2d(&tmap_x, x, y);
      tma_prefetch_2d(&tmap_x, a.N + x, y);
    }
  }
  __syncthreads();
  const bool ok = mbar_wait_bounded(bar, 0, a.timeout_ns);
  if (__syncthreads_or(!ok)) {
    if (tid == 0) {
      if (a.dev_err) atomicOr(a.dev_err, MXQ_DEVERR_TIMEOUT);
      mbar_wait_bounded(bar, 0, a.timeout_ns);
    }
    return;
  }
  const int rl = 2 * SAVE_LR * warp + SAVE_LR * h;
  const int width = min(MX_TILE_K, a.N - col0);
  const bool mine = row0 + rl < a.M && 8 * c < width;
  const uint32_t ceil_bf16 = a.scale_ceil ? 0x001F001Fu : 0u;
  const uint32_t src = sbase + rl * BF16_PITCH + c * 16;
  const int64_t pitch = 2 * static_cast<int64_t>(a.N);
  uint8_t* q = a.x_q + (row0 + rl) * pitch + col0 + 8 * c;
  // The checkpoint's halves one after the other, then both again for the activation:
  // 16 registers instead of 32 across the first two.
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    uint32_t v[SAVE_LR][4];
#pragma unroll
    for (int i = 0; i < SAVE_LR; ++i) {
      const uint4 x = lds128(src + half * L::UP + i * BF16_PITCH);
      v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
    }
    save_block(v, q + half * a.N, pitch, mine, sbase + L::SAVED + half * 4 * TILE_ROWS, rl, c,
               ceil_bf16);
  }
  float y[SAVE_LR][8];
#pragma unroll
  for (int i = 0; i < SAVE_LR; ++i) {
    const uint4 vg = lds128(src + i * BF16_PITCH), vu = lds128(src + L::UP + i * BF16_PITCH);
    const uint32_t g[4] = {vg.x, vg.y, vg.z, vg.w}, u[4] = {vu.x, vu.y, vu.z, vu.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      // Columns past N hold other values of x; scale tiles are padded with zeros.
      const float2 z = 8 * c < width ? gate_pair<GELU>(pair_of(g[p]), pair_of(u[p])) : f2(0.0f);
      y[i][2 * p] = z.x;
      y[i][2 * p + 1] = z.y;
    }
  }
  TileOut o{};
  o.M = a.M;
  o.pitch = a.N;
  o.row0 = row0;
  o.col0 = col0;
  o.width = width;
  o.q_row = a.q_row;
  o.s_row = a.s_row;
  o.s_col = a.s_col;
  o.q_col = &tmap_qcol;
  o.qcol_x = row0;
  o.qcol_y = col0 / 8;
  o.tiled = a.scale_tiled;
  quantize_tile<SAVE_LR, (MODE & MX_ROW) != 0, (MODE & MX_COL) != 0>(
      y, tile_shared(sbase, sbase + L::SCALES), o, a.scale_ceil ? 0x001FFFFFu : 0u);
  // The checkpoint's scales, staged before quantize_tile's barriers: the first half
  // of the threads the gate's, the others the up's.
  const int64_t ld = pitch / 32;
#pragma unroll
  for (int half = 0; half < 2; ++half)
    store_row_scales<Tile<SAVE_LR>::THREADS>(
        sbase + L::SAVED + half * (4 * TILE_ROWS), min(TILE_ROWS, a.M - row0),
        a.x_s + row0 * ld + (half * a.N + col0) / 32, ld, a.N % 128 == 0, width / 32,
        (tid + half * TILE_ROWS) % Tile<SAVE_LR>::THREADS);
  if (tid == 0) bulk_wait_read<0>();
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

struct DGatedSavedShared {
  static constexpr int GATE = BF16_TILE;                 // codes
  static constexpr int UP = GATE + CODE_TILE;
  static constexpr int STAGING = UP + CODE_TILE;         // colwise codes
  static constexpr int SCALES = STAGING + TILE_CODES_BYTES;
  static constexpr int SAVED = SCALES + Tile<BACK_LR>::SCALES_BYTES;   // [2][rows][4] fp32
  static constexpr int DYNAMIC = SAVED + 32 * TILE_ROWS + 1024;       // + alignment pad
};

// act(x) and act'(x) of silu or gelu_tanh from one sigmoid, s = 1 / (1 + e):
//   silu, e = e^-x:      value v = x s,  slope s (1 + x (1 - s)) = s + s (x - v);
//   gelu_tanh, e = e^-2u with u = sqrt(2/pi) (x + 0.044715 x^3), (1 + tanh u) / 2 = s:
//                        value v = x s,  slope s + s (x - v) 2 u'.
// e may overflow: s is then 0, and so are both.  x - v cancels where s is near 1, to
// 2^-22 of x; from x = 18 on (4.5 for gelu) s is 1 and x - v nothing, so that the slope
// is off by 2^-17 at most.  Nine and sixteen instructions a pair; forms from e^-|x|,
// which select by the sign of x, take twenty and thirty.
template <bool GELU>
__device__ __forceinline__ void act_pair_d(float2 x, float2& value, float2& slope) {
  constexpr float kLog2e = 1.4426950408889634f, kC = 0.7978845608028654f;
  float2 x2, arg;
  if constexpr (GELU) {
    // Cut off far above where s is 0 or 1, so that s (x - v) = 0 times it is 0.
    x2 = mul_f32x2(x, x);
    x2 = make_float2(fminf(x2.x, 1e30f), fminf(x2.y, 1e30f));
    arg = mul_f32x2(x, fma_f32x2(x2, f2(-2.0f * kC * kLog2e * 0.044715f), f2(-2.0f * kC * kLog2e)));
  } else {
    arg = mul_f32x2(x, f2(-kLog2e));
  }
  const float2 s = rcp_pair(add_f32x2(ex2_pair(arg), f2(1.0f)));
  value = mul_f32x2(x, s);
  const float2 rest = fma_f32x2(value, f2(-1.0f), x);
  if constexpr (GELU)
    slope = fma_f32x2(mul_f32x2(s, rest), fma_f32x2(x2, f2(2.0f * kC * 3.0f * 0.044715f), f2(2.0f * kC)), s);
  else
    slope = fma_f32x2(s, rest, s);
}

// Eight E4M3 codes (two words) times a scale.
__device__ __forceinline__ void decode8(uint2 q, float scale, float2 (&v)[4]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w[p]));
    v[2 * p] = mul_f32x2(__half22float2(*reinterpret_cast<const __half2*>(&lo)), f2(scale));
    v[2 * p + 1] = mul_f32x2(__half22float2(*reinterpret_cast<const __half2*>(&hi)), f2(scale));
  }
}

// 2^(code - 127); 255 is NaN.
__device__ __forceinline__ uint32_t e8m0_bits(uint32_t code) {
  return code == 255u ? 0x7FC00000u : code == 0u ? 0x00400000u : code << 23;
}

template <int MODE, bool GELU>
__global__ void __launch_bounds__(Tile<BACK_LR>::THREADS, CTAS)
mx_dgated_saved_kernel(const __grid_constant__ CUtensorMap tmap_grad,
                       const __grid_constant__ CUtensorMap tmap_saved,
                       const __grid_constant__ CUtensorMap tmap_qcol,
                       const __grid_constant__ CUtensorMap tmap_qcol2, const SavedArgs a) {
  using L = DGatedSavedShared;
  constexpr bool ROW = (MODE & MX_ROW) != 0, COL = (MODE & MX_COL) != 0;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full;
  const uint32_t sbase = smem_addr(align_up_shared<1024>(smem_raw));
  const uint32_t bar = smem_addr(&full);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = lane >> 4, c = lane & 15;
  const int band = static_cast<int>(blockIdx.x) / a.tiles_k;
  const int tk = static_cast<int>(blockIdx.x) - band * a.tiles_k;
  const int row0 = band * TILE_ROWS, col0 = tk * MX_TILE_K;
  const int width = min(MX_TILE_K, a.N - col0);
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
    mbar_arrive_expect_tx(bar, BF16_TILE + 2 * CODE_TILE);
    tma_load_2d(sbase, &tmap_grad, col0, row0, bar);
    tma_load_2d(sbase + L::GATE, &tmap_saved, col0, row0, bar);
    tma_load_2d(sbase + L::UP, &tmap_saved, a.N + col0, row0, bar);
  }
  // The checkpoint's scales of the tile, four bytes a row: the gate's, then the up's.
  const int64_t ld = 2 * static_cast<int64_t>(a.N) / 32;
  for (int i = tid; i < 2 * TILE_ROWS; i += Tile<BACK_LR>::THREADS) {
    const int half = i / TILE_ROWS, line = i % TILE_ROWS;
    uint32_t v = 0;
    if (row0 + line < a.M) {
      const uint8_t* p = a.saved_s + (row0 + line) * ld + (half * a.N + col0) / 32;
      if (width == MX_TILE_K && (reinterpret_cast<uintptr_t>(p) & 3u) == 0) {
        v = *reinterpret_cast<const uint32_t*>(p);
      } else {
        for (int b = 0; b < width / 32; ++b) v |= static_cast<uint32_t>(p[b]) << (8 * b);
      }
    }
    sts128(sbase + L::SAVED + 16 * i, e8m0_bits(v & 0xFFu), e8m0_bits(v >> 8 & 0xFFu),
           e8m0_bits(v >> 16 & 0xFFu), e8m0_bits(v >> 24));
  }
  __syncthreads();
  const bool ok = mbar_wait_bounded(bar, 0, a.timeout_ns);
  if (__syncthreads_or(!ok)) {
    if (tid == 0) {
      if (a.dev_err) atomicOr(a.dev_err, MXQ_DEVERR_TIMEOUT);
      mbar_wait_bounded(bar, 0, a.timeout_ns);
    }
    return;
  }
  const int rl = 2 * BACK_LR * warp + BACK_LR * h;
  const uint32_t grad_at = sbase + rl * BF16_PITCH + c * 16;
  const uint32_t gate_at = sbase + L::GATE + rl * MX_TILE_K + c * 8;
  const uint32_t up_at = gate_at + CODE_TILE;
  const uint32_t scale_at = sbase + L::SAVED + rl * 16 + (c >> 2) * 4;
  const uint32_t ceil_f32 = a.scale_ceil ? 0x001FFFFFu : 0u;
  float y[BACK_LR][8];
  // d gate, with d up parked as fp32 in the bytes of this lane's own operands.
#pragma unroll
  for (int i = 0; i < BACK_LR; ++i) {
    const uint4 gv = lds128(grad_at + i * BF16_PITCH);
    const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
    float2 gate[4], up[4], park[4];
    decode8(lds64(gate_at + i * MX_TILE_K), __uint_as_float(lds32(scale_at + 16 * i)), gate);
    decode8(lds64(up_at + i * MX_TILE_K), __uint_as_float(lds32(scale_at + 16 * TILE_ROWS + 16 * i)), up);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float2 value, slope;
      act_pair_d<GELU>(gate[p], value, slope);
      const float2 grad = pair_of(gw[p]);
      const float2 dg = mul_f32x2(mul_f32x2(grad, up[p]), slope);
      park[p] = mul_f32x2(grad, value);
      y[i][2 * p] = dg.x;
      y[i][2 * p + 1] = dg.y;
    }
    sts128(grad_at + i * BF16_PITCH, __float_as_uint(park[0].x), __float_as_uint(park[0].y),
           __float_as_uint(park[1].x), __float_as_uint(park[1].y));
    sts64(gate_at + i * MX_TILE_K, __float_as_uint(park[2].x), __float_as_uint(park[2].y));
    sts64(up_at + i * MX_TILE_K, __float_as_uint(park[3].x), __float_as_uint(park[3].y));
  }
  TileOut o{};
  o.M = a.M;
  o.pitch = 2 * static_cast<int64_t>(a.N);
  o.row0 = row0;
  o.col0 = col0;
  o.width = width;
  o.q_row = a.q_row;
  o.s_row = a.s_row;
  o.s_col = a.s_col;
  o.q_col = &tmap_qcol;
  o.qcol_x = row0;
  o.qcol_y = col0 / 8;
  o.tiled = a.scale_tiled;
  quantize_tile<BACK_LR, ROW, COL>(y, tile_shared(sbase + L::STAGING, sbase + L::SCALES), o, ceil_f32);
#pragma unroll
  for (int i = 0; i < BACK_LR; ++i) {
    const uint4 lo = lds128(grad_at + i * BF16_PITCH);
    const uint2 mid = lds64(gate_at + i * MX_TILE_K), hi = lds64(up_at + i * MX_TILE_K);
    y[i][0] = __uint_as_float(lo.x); y[i][1] = __uint_as_float(lo.y);
    y[i][2] = __uint_as_float(lo.z); y[i][3] = __uint_as_float(lo.w);
    y[i][4] = __uint_as_float(mid.x); y[i][5] = __uint_as_float(mid.y);
    y[i][6] = __uint_as_float(hi.x); y[i][7] = __uint_as_float(hi.y);
  }
  o.col0 = a.N + col0;
  o.q_col = &tmap_qcol2;
  // By the call's first barrier every lane has read its parked values: the gradient's
  // tile is the second staging, and the first one's store is not waited for.
  quantize_tile<BACK_LR, ROW, COL>(y, tile_shared(sbase, sbase + L::SCALES), o, ceil_f32);
  if (tid == 0) bulk_wait_read<0>();
}

template <int MODE, bool GELU>
cudaError_t gated_save(const SavedMaps& maps, const SavedArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  auto kernel = mx_gated_save_kernel<MODE, GELU>;
  cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), GatedSaveShared::DYNAMIC, &allowed);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((a.M + TILE_ROWS - 1) / TILE_ROWS) * a.tiles_k;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  kernel<<<static_cast<unsigned>(tiles), Tile<SAVE_LR>::THREADS, GatedSaveShared::DYNAMIC, stream>>>(maps.a, maps.q_col, a);
  return cudaGetLastError();
}

template <int MODE, bool GELU>
cudaError_t dgated_saved(const SavedMaps& maps, const SavedArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  auto kernel = mx_dgated_saved_kernel<MODE, GELU>;
  cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), DGatedSavedShared::DYNAMIC, &allowed);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((a.M + TILE_ROWS - 1) / TILE_ROWS) * a.tiles_k;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  kernel<<<static_cast<unsigned>(tiles), Tile<BACK_LR>::THREADS, DGatedSavedShared::DYNAMIC, stream>>>(
      maps.a, maps.b, maps.q_col, maps.q_col2, a);
  return cudaGetLastError();
}

}  // namespace

int saved_tile_rows() { return TILE_ROWS; }
int saved_prefetch(int num_sms) { return num_sms * CTAS / 2; }

cudaError_t launch_gated_save(const SavedMaps& maps, const SavedArgs& a, int mode, bool gelu,
                              cudaStream_t stream) {
  switch (mode) {
    case MX_ROW: return gelu ? gated_save<MX_ROW, true>(maps, a, stream) : gated_save<MX_ROW, false>(maps, a, stream);
    case MX_COL: return gelu ? gated_save<MX_COL, true>(maps, a, stream) : gated_save<MX_COL, false>(maps, a, stream);
    default: return gelu ? gated_save<MX_ROW | MX_COL, true>(maps, a, stream)
                         : gated_save<MX_ROW | MX_COL, false>(maps, a, stream);
  }
}

cudaError_t launch_dgated_saved(const SavedMaps& maps, const SavedArgs& a, int mode, bool gelu,
                                cudaStream_t stream) {
  switch (mode) {
    case MX_ROW: return gelu ? dgated_saved<MX_ROW, true>(maps, a, stream) : dgated_saved<MX_ROW, false>(maps, a, stream);
    case MX_COL: return gelu ? dgated_saved<MX_COL, true>(maps, a, stream) : dgated_saved<MX_COL, false>(maps, a, stream);
    default: return gelu ? dgated_saved<MX_ROW | MX_COL, true>(maps, a, stream)
                         : dgated_saved<MX_ROW | MX_COL, false>(maps, a, stream);
  }
}

}  // namespace mxq
