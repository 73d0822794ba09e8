// rmsnorm_kernels.cu -- RMSNorm with the residual's addition and MXFP8 output,
// and its backward pass.
//
//   h = bf16(x + residual),  rstd = (mean h^2 + eps)^(-1/2),  y = (h rstd) weight
//
// Rows (rmsnorm_rows_kernel): a row's values stay in the registers of the threads
// that loaded them, packed as bf16, so that h, rstd, y and its rowwise codes and
// scales come from one read of the inputs.  Sixteen values a thread in one 32-byte
// access: a block's scale takes one exchange between lanes instead of two for half the
// values, and the sum of bf16 pairs one instruction instead of six.  16384 x 8192 with
// a residual 136 us, 6.95 TB/s (1.02 of the copy rate, measured); in 16-byte vectors
// with fp32 additions 171 us.
// Columns (rmsnorm_cols_kernel): a column's block of 32 rows needs the rstd of all
// of them, so that the colwise codes are a second pass over h: 193 us with both, where
// the bytes of two passes take 199 and those of one 160.  Not kept: both passes in one
// grid, tiles a few bands behind the rows whose h they find in L2 (199 us at best: the
// rows' CTAs then have the tiles' registers, and too few are resident), and the two
// passes by turns over chunks that fit L2 (220 us for 64 MB, 243 for 16: the column pass
// is no faster from L2), and one pass by clusters of 16 CTAs that hold 64 rows in shared
// memory and exchange their sums (251 us: loading, the barrier and the codes of a CTA come
// one after another).
// Backward (rmsnorm_back_kernel): with g = dy weight and c = rstd^2 mean(g h),
//   dx = dh + rstd (g - h c),   dweight = sum over the rows of dy (h rstd).
// Rows come by bulk copies into a ring of shared memory, so that what is under way does
// not depend on the registers that the columns' sums leave: 16384 x 8192 157 us, 6.85 TB/s
// (1.01); with loads into registers, two CTAs of 256 threads an SM, 172 us, and where those
// fill worse 9830 x 10240 176 us against 117.

#include "mx_elements.cuh"
#include "mx_tile.cuh"
#include "mxq_internal.h"
#include "mxq_layer.h"
#include "mxq_products.h"
#include "mxq_ptx.cuh"

namespace mxq {
namespace {

__device__ __forceinline__ uint4 ldg128_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(v.y), "f"(v.x));
  return d;
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t v) {
  return make_float2(bf16_lo(v), bf16_hi(v));
}

// x + y of two pairs, each rounded once (the sum of two bf16 values that could
// round otherwise fits in fp32 exactly, so this is also bf16(fp32 sum)).
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}

// Sixteen bf16 values, 32 bytes: in one access where the address allows (`wide`).
struct Granule {
  uint32_t u[8];
};

__device__ __forceinline__ Granule load_granule(const uint16_t* p, bool wide) {
  Granule g;
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(g.u[0]), "=r"(g.u[1]), "=r"(g.u[2]), "=r"(g.u[3]), "=r"(g.u[4]),
                   "=r"(g.u[5]), "=r"(g.u[6]), "=r"(g.u[7]) : "l"(p));
  } else {
    const uint4 a = ldg128_stream(p), b = ldg128_stream(p + 8);
    g.u[0] = a.x; g.u[1] = a.y; g.u[2] = a.z; g.u[3] = a.w;
    g.u[4] = b.x; g.u[5] = b.y; g.u[6] = b.z; g.u[7] = b.w;
  }
  return g;
}

__device__ __forceinline__ void store_granule(uint16_t* p, const Granule& g, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(g.u[0]), "r"(g.u[1]), "r"(g.u[2]), "r"(g.u[3]), "r"(g.u[4]),
                    "r"(g.u[5]), "r"(g.u[6]), "r"(g.u[7]) : "memory");
  } else {
    stg128(p, g.u[0], g.u[1], g.u[2], g.u[3]);
    stg128(p + 8, g.u[4], g.u[5], g.u[6], g.u[7]);
  }
}

// Eight weights from column `k` on, as pairs.
__device__ __forceinline__ void load_weight(const void* weight, int f32, int k, float2 (&w)[4]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(weight) + k);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    w[0] = make_float2(a.x, a.y);
    w[1] = make_float2(a.z, a.w);
    w[2] = make_float2(b.x, b.y);
    w[3] = make_float2(b.z, b.w);
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(weight) + k));
    w[0] = unpack_bf16(a.x);
    w[1] = unpack_bf16(a.y);
    w[2] = unpack_bf16(a.z);
    w[3] = unpack_bf16(a.w);
  }
}

// The sum of a row: v[i] is the sum of this lane's granule i * 32 * WARPS + t.
// Always grouped alike -- 32 neighbouring granules by a butterfly, then those sums in
// four interleaved chains -- so that the bits depend on the row alone and not on how
// many warps hold it (granules past the row add +0 to sums that are not -0).  `part`
// holds WARPS * VPT floats of this row.
template <int WARPS, int VPT>
__device__ __forceinline__ float row_sum(float (&v)[VPT], float* part, int warp) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  if constexpr (WARPS == 1 && VPT == 1) return v[0];
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) part[i * WARPS + warp] = v[i];
  }
  __syncthreads();
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < WARPS * VPT; ++j) s[j & 3] += part[j];
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// One row by the 32 * WARPS threads that call this with t = 0 .. 32 * WARPS - 1; a
// thread holds VPT granules of sixteen values, so that a block of 32 is in two
// neighbouring lanes.  Rows past M (padding of scale tiles) write zeros to s_row.
template <int WARPS, int VPT>
__device__ __forceinline__ void norm_row(const NormArgs& a, int64_t row, int t, float* part) {
  constexpr int THREADS = 32 * WARPS;
  const int granules = a.K / 16;
  const bool real = row < a.M;
  Granule v[VPT];
  float sums[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) sums[i] = 0.0f;
  if (real) {
    const uint16_t* px = a.x + row * a.ldx;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int n = i * THREADS + t;
      if (n < granules) v[i] = load_granule(px + 16 * n, a.wide & 1);
    }
    if (a.residual) {
      const uint16_t* pr = a.residual + row * a.ldr;
      Granule r[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int n = i * THREADS + t;
        if (n < granules) r[i] = load_granule(pr + 16 * n, a.wide & 2);
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int p = 0; p < 8; ++p) v[i].u[p] = add_bf16x2(v[i].u[p], r[i].u[p]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * THREADS + t < granules) {
        float2 sum = f2(0.0f);
#pragma unroll
        for (int p = 0; p < 8; ++p)
          sum = fma_f32x2(unpack_bf16(v[i].u[p]), unpack_bf16(v[i].u[p]), sum);
        sums[i] = sum.x + sum.y;
      }
    if (a.h) {
      uint16_t* ph = a.h + row * a.ldh;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int n = i * THREADS + t;
        if (n < granules) store_granule(ph + 16 * n, v[i], a.wide & 4);
      }
    }
  }
  const float ss = row_sum<WARPS, VPT>(sums, part, t / 32);
  const float rstd = __frsqrt_rn(fmaf(ss, a.inv_k, a.eps));
  if (real && t == 0) a.rstd[row] = rstd;
  if (!a.y && !a.q_row) return;

  const uint32_t ceil_f32 = a.scale_ceil ? 0x001FFFFFu : 0u;
  const int nkb = a.K / 32;
  const int lane = t & 31;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int n = i * THREADS + t;
    // Lanes in pairs have granules or not, and in eights there is one at least
    // where there is a word of scales to write.
    const bool in = n < granules;
    float2 y[8];
    if (in && real) {
      float2 w[8];
      load_weight(a.weight, a.weight_f32, 16 * n, reinterpret_cast<float2(&)[4]>(w[0]));
      load_weight(a.weight, a.weight_f32, 16 * n + 8, reinterpret_cast<float2(&)[4]>(w[4]));
#pragma unroll
      for (int p = 0; p < 8; ++p)
        y[p] = mul_f32x2(mul_f32x2(unpack_bf16(v[i].u[p]), f2(rstd)), w[p]);
      if (a.y) {
        Granule o;
#pragma unroll
        for (int p = 0; p < 8; ++p) o.u[p] = pack_bf16(y[p]);
        store_granule(a.y + row * a.ldy + 16 * n, o, a.wide & 8);
      }
    }
    if (a.q_row) {
      uint32_t code = 0u;
      uint32_t e = 0u;
      if (in && real) {
        float m = fmaxf(fabsf(y[0].x), fabsf(y[0].y));
#pragma unroll
        for (int p = 1; p < 8; ++p) m = fmax3(m, fabsf(y[p].x), fabsf(y[p].y));
        e = f32_scale_exponent(__float_as_uint(m), ceil_f32);
      }
      e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 1));
      if (in && real) {
        code = e8m0_from_exponent(e);
        const float inv = inv_scale_from_e8m0(code);
        uint32_t q[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const float2 z = mul_f32x2(y[p], f2(inv));
          q[p] = cvt_e4m3x2(z.x, z.y);
        }
        stg128_cs(a.q_row + row * a.K + 16 * n, q[0] | (q[1] << 16), q[2] | (q[3] << 16),
                  q[4] | (q[5] << 16), q[6] | (q[7] << 16));
      }
      // The scales of eight lanes' four blocks as one word.
      uint32_t word = code << (8 * ((lane >> 1) & 3));
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
      const int kb = n / 2;             // this lane's block
      if (a.scale_tiled) {
        if ((lane & 7) == 0 && in && row < a.rows)
          stg32(a.s_row + ((row >> 7) * ((nkb + 3) / 4) + (kb >> 2)) * 512 + (row & 31) * 16 +
                    ((row & 127) >> 5) * 4,
                word);
      } else if (real) {
        if ((nkb & 3) == 0) {
          if ((lane & 7) == 0 && in) stg32(a.s_row + row * nkb + kb, word);
        } else if ((lane & 1) == 0 && in) {
          stg8(a.s_row + row * nkb + kb, code);
        }
      }
    }
  }
}

// A CTA takes a row, or several in four warps at most.
template <int WARPS>
constexpr int norm_rows_per_cta() { return WARPS >= 4 ? 1 : 4 / WARPS; }

template <int WARPS, int VPT>
__global__ void __launch_bounds__(32 * WARPS * norm_rows_per_cta<WARPS>())
rmsnorm_rows_kernel(const NormArgs a) {
  constexpr int ROWS = norm_rows_per_cta<WARPS>();
  __shared__ float part[ROWS][WARPS * VPT];
  grid_launch_dependents();
  const int sub = ROWS == 1 ? 0 : threadIdx.x / (32 * WARPS);
  const int t = ROWS == 1 ? threadIdx.x : threadIdx.x % (32 * WARPS);
  norm_row<WARPS, VPT>(a, static_cast<int64_t>(blockIdx.x) * ROWS + sub, t, part[sub]);
}

// ---------------------------------------------------------------------------
// Colwise codes
// ---------------------------------------------------------------------------

// Eight rows a lane and six CTAs an SM (80 registers): 16384 x 8192 takes 61 us behind
// the row pass, with five CTAs 66 us, with seven, which spill, 73 us, with four rows a
// lane 77 us (the pass computes little, and pays for exchanges among more warps).
constexpr int LR = 8;
constexpr int TILE_THREADS = Tile<LR>::THREADS;
constexpr int TILE_SCALES_BYTES = Tile<LR>::SCALES_BYTES;
constexpr int COL_CTAS = 6;      // an SM
// A CTA has the tile half a wave on (COL_CTAS / 2 an SM) brought into L2: 192.4 us with the
// row pass instead of 197.4 (a quarter of a wave 193.6, a whole one 193.2).
constexpr int COL_TILE_BYTES = TILE_ROWS * MX_TILE_K * 2;
constexpr int COL_SHARED = COL_TILE_BYTES + TILE_SCALES_BYTES;

__global__ void __launch_bounds__(TILE_THREADS, COL_CTAS)
rmsnorm_cols_kernel(const __grid_constant__ CUtensorMap tmap_h,
                    const __grid_constant__ CUtensorMap tmap_qcol, const NormArgs a,
                    uint8_t* s_col, int tiles_k, int ahead, uint32_t* dev_err,
                    uint64_t timeout_ns) {
  __shared__ __align__(1024) uint8_t smem[COL_SHARED];
  __shared__ __align__(8) uint64_t full;
  const uint32_t sbase = smem_addr(smem), bar = smem_addr(&full);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = lane >> 4, c = lane & 15;
  // Last band first: those rows of h are still in L2.
  const int tile = static_cast<int>(gridDim.x - 1 - blockIdx.x);
  const int band = tile / tiles_k;
  const int row0 = band * TILE_ROWS, col0 = (tile - band * tiles_k) * MX_TILE_K;
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  grid_dependency_wait();   // rstd and h of the row pass
  if (tid == 0) {
    mbar_arrive_expect_tx(bar, COL_TILE_BYTES);
    tma_load_2d(sbase, &tmap_h, col0, row0, bar);
    if (tile >= ahead)
      tma_prefetch_2d(&tmap_h, (tile - ahead) % tiles_k * MX_TILE_K, (tile - ahead) / tiles_k * TILE_ROWS);
  }
  float2 w[4];
  if (col0 + 8 * c < a.K) load_weight(a.weight, a.weight_f32, col0 + 8 * c, w);
  else w[0] = w[1] = w[2] = w[3] = f2(0.0f);
  float r[LR];
  const int rl = 2 * LR * warp + LR * h;
#pragma unroll
  for (int i = 0; i < LR; i += 4) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row0 + rl < a.M) v = *reinterpret_cast<const float4*>(a.rstd + row0 + rl + i);
    r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
  }
  __syncthreads();
  const bool ok = mbar_wait_bounded(bar, 0, timeout_ns);
  float y[LR][8];
  const uint32_t src = sbase + rl * (MX_TILE_K * 2) + c * 16;
#pragma unroll
  for (int i = 0; i < LR; ++i) {
    const uint4 v = ok ? lds128(src + i * (MX_TILE_K * 2)) : make_uint4(0, 0, 0, 0);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 z = mul_f32x2(mul_f32x2(unpack_bf16(u[p]), f2(r[i])), w[p]);
      y[i][2 * p] = z.x;
      y[i][2 * p + 1] = z.y;
    }
  }
  // The tile has been read by every warp: it becomes the staging.
  if (__syncthreads_or(!ok)) {
    if (tid == 0) {
      if (dev_err) atomicOr(dev_err, MXQ_DEVERR_TIMEOUT);
      mbar_wait_bounded(bar, 0, timeout_ns);
    }
    return;
  }
  TileOut o{};
  o.M = a.M;
  o.pitch = a.K;
  o.row0 = row0;
  o.col0 = col0;
  o.width = min(MX_TILE_K, a.K - col0);
  o.s_col = s_col;
  o.q_col = &tmap_qcol;
  o.qcol_x = row0;
  o.qcol_y = col0 / 8;
  o.tiled = a.scale_tiled;
  quantize_tile<LR, false, true>(y, tile_shared(sbase, sbase + COL_TILE_BYTES), o,
                                        a.scale_ceil ? 0x001FFFFFu : 0u);
  if (tid == 0) bulk_wait_read<0>();
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// 32 * WARPS threads walk over the rows blockIdx.x, blockIdx.x + gridDim.x, ... with the
// columns' sums in registers, VECS vectors of eight values a thread.  Rows arrive in a
// ring of shared memory, as many ahead as it holds.  dy and h go into registers in one
// go (KEEP), so that the barrier of the row's sum frees their place for a later row; dh
// is read from its place behind it, and that is free at the next row's barrier.  Where
// the registers do not hold a row, both are read twice and a second barrier frees them.
constexpr int BACK_STAGES = 4;

template <int WARPS, int VECS, bool W32, bool KEEP>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS)
rmsnorm_back_kernel(const NormBackArgs a, int stages) {
  constexpr int THREADS = 32 * WARPS;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float part[2][WARPS];
  __shared__ __align__(8) uint64_t bars[2 * BACK_STAGES];
  grid_launch_dependents();
  const int t = threadIdx.x, vectors = a.K / 8;
  const uint32_t bytes = 2 * a.K, slot = bytes * (a.dh ? 3 : 2);
  const uint32_t base = smem_addr(ring), main = smem_addr(bars), past = main + 8 * BACK_STAGES;
  const int rows = (a.M - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1;
  auto row_of = [&](int i) { return blockIdx.x + static_cast<int64_t>(i) * gridDim.x; };
  // Row i into place s, by one thread.
  auto load_main = [&](int i, int s) {
    if (i >= rows) return;
    mbar_arrive_expect_tx(main + 8 * s, 2 * bytes);
    bulk_load(base + s * slot, a.dy + row_of(i) * a.lddy, bytes, main + 8 * s);
    bulk_load(base + s * slot + bytes, a.h + row_of(i) * a.ldh, bytes, main + 8 * s);
  };
  auto load_past = [&](int i, int s) {
    if (i >= rows || !a.dh) return;
    mbar_arrive_expect_tx(past + 8 * s, bytes);
    bulk_load(base + s * slot + 2 * bytes, a.dh + row_of(i) * a.lddh, bytes, past + 8 * s);
  };
  if (t == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(main + 8 * s, 1);
      mbar_init(past + 8 * s, 1);
    }
    fence_barrier_init();
    for (int s = 0; s < stages; ++s) {
      load_main(s, s);
      load_past(s, s);
    }
  }
  float2 dw[VECS][4], kept32[W32 && KEEP ? VECS : 1][4];
  uint4 kept16[!W32 && KEEP ? VECS : 1];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
#pragma unroll
    for (int p = 0; p < 4; ++p) dw[i][p] = f2(0.0f);
    if (KEEP && i * THREADS + t < vectors) {
      if constexpr (W32)
        load_weight(a.weight, 1, 8 * (i * THREADS + t), kept32[KEEP ? i : 0]);
      else
        kept16[KEEP ? i : 0] = __ldg(static_cast<const uint4*>(a.weight) + i * THREADS + t);
    }
  }
  auto weight_of = [&](int i, float2 (&w)[4]) {
    if constexpr (!KEEP) {
      load_weight(a.weight, W32, 8 * (i * THREADS + t), w);
    } else if constexpr (W32) {
#pragma unroll
      for (int p = 0; p < 4; ++p) w[p] = kept32[i][p];
    } else {
      w[0] = unpack_bf16(kept16[i].x);
      w[1] = unpack_bf16(kept16[i].y);
      w[2] = unpack_bf16(kept16[i].z);
      w[3] = unpack_bf16(kept16[i].w);
    }
  };
  float rstd = a.rstd[blockIdx.x];
  __syncthreads();

  bool ok = true;
  int s = 0, before = 0, i = 0;
  uint32_t phase = 0;
  for (; i < rows; ++i) {
    ok = mbar_wait_bounded(main + 8 * s, phase, a.timeout_ns) && ok;
    const uint32_t mine = base + s * slot + 16 * t;
    uint4 dy[KEEP ? VECS : 1], h[KEEP ? VECS : 1];
    float2 sum = f2(0.0f);
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      if (v * THREADS + t >= vectors) continue;
      const int at = KEEP ? v : 0;
      dy[at] = lds128(mine + v * THREADS * 16);
      h[at] = lds128(mine + v * THREADS * 16 + bytes);
      const uint32_t ud[4] = {dy[at].x, dy[at].y, dy[at].z, dy[at].w};
      const uint32_t uh[4] = {h[at].x, h[at].y, h[at].z, h[at].w};
      float2 w[4];
      weight_of(v, w);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 d = unpack_bf16(ud[p]);
        const float2 n = mul_f32x2(unpack_bf16(uh[p]), f2(rstd));
        dw[v][p] = fma_f32x2(d, n, dw[v][p]);
        sum = fma_f32x2(mul_f32x2(d, w[p]), n, sum);
      }
    }
    float c = sum.x + sum.y;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, d);
    if constexpr (WARPS > 1) {
      if ((t & 31) == 0) part[i & 1][t >> 5] = c;
      if (__syncthreads_or(!ok)) break;
      float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < WARPS; ++j) sums[j & 3] += part[i & 1][j];
      c = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    } else if (__any_sync(0xFFFFFFFFu, !ok)) {
      break;
    }
    c *= a.inv_k;
    if (t == 0 && KEEP) {
      load_main(i + stages, s);
      if (i > 0) load_past(i - 1 + stages, before);
    }
    const float scale = rstd;
    if (i + 1 < rows) rstd = a.rstd[row_of(i + 1)];
    if (a.dh) ok = mbar_wait_bounded(past + 8 * s, phase, a.timeout_ns);
    uint16_t* dx = a.dx + row_of(i) * a.lddx + 8 * t;
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      if (v * THREADS + t >= vectors) continue;
      uint4 yv, hv, r = make_uint4(0, 0, 0, 0);
      if constexpr (KEEP) {
        yv = dy[v];
        hv = h[v];
      } else {
        yv = lds128(mine + v * THREADS * 16);
        hv = lds128(mine + v * THREADS * 16 + bytes);
      }
      if (a.dh) r = lds128(mine + v * THREADS * 16 + 2 * bytes);
      const uint32_t ud[4] = {yv.x, yv.y, yv.z, yv.w}, uh[4] = {hv.x, hv.y, hv.z, hv.w};
      const uint32_t ur[4] = {r.x, r.y, r.z, r.w};
      uint32_t o[4];
      float2 w[4];
      weight_of(v, w);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 n = mul_f32x2(unpack_bf16(uh[p]), f2(scale));
        const float2 g = mul_f32x2(unpack_bf16(ud[p]), w[p]);
        o[p] = pack_bf16(fma_f32x2(fma_f32x2(n, f2(-c), g), f2(scale), unpack_bf16(ur[p])));
      }
      stg128(dx + v * THREADS * 8, o[0], o[1], o[2], o[3]);
    }
    if constexpr (!KEEP) {
      __syncthreads();
      if (t == 0) {
        load_main(i + stages, s);
        load_past(i + stages, s);
      }
    }
    before = s;
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
  if (__syncthreads_or(i < rows || !ok)) {
    // A copy did not arrive.  Those under way end before the CTA does, or time out too.
    if (t == 0) {
      if (a.dev_err) atomicOr(a.dev_err, MXQ_DEVERR_TIMEOUT);
      for (int j = i; j < min(i + stages, rows); ++j)
        mbar_wait_bounded(main + 8 * (j % stages), j / stages & 1, a.timeout_ns);
      for (int j = max(i - 1, 0); a.dh && j < min(i - (KEEP ? 1 : 0) + stages, rows); ++j)
        mbar_wait_bounded(past + 8 * (j % stages), j / stages & 1, a.timeout_ns);
    }
    return;
  }
  if (!a.parts) return;
  float* out = a.parts + static_cast<int64_t>(blockIdx.x) * a.K + 8 * t;
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    if (v * THREADS + t >= vectors) continue;
    float4* p = reinterpret_cast<float4*>(out + v * THREADS * 8);
    p[0] = make_float4(dw[v][0].x, dw[v][0].y, dw[v][1].x, dw[v][1].y);
    p[1] = make_float4(dw[v][2].x, dw[v][2].y, dw[v][3].x, dw[v][3].y);
  }
}

// dweight[k] = sum over the CTAs' column sums.  A block takes 16 columns: thread (g, q)
// adds columns 4q .. 4q + 3 of the parts g, g + 128, ..., and the 128 sums are added in a
// fixed tree.  (16384 x 256 has 2432 parts: with the columns before 11.5 us, with 32
// columns a block 13.3 and with 8 10.8; 12288 x 8192 118.8, 119.0 and 120.2.)
constexpr int DW_QUADS = 4, DW_GROUPS = 128;
__global__ void __launch_bounds__(DW_QUADS * DW_GROUPS)
rmsnorm_dweight_kernel(const float* __restrict__ parts, int count, int K, float* __restrict__ dweight) {
  __shared__ float4 s[DW_GROUPS][DW_QUADS];
  grid_dependency_wait();
  const int q = threadIdx.x % DW_QUADS, g = threadIdx.x / DW_QUADS;
  const float* p = parts + blockIdx.x * (4 * DW_QUADS) + 4 * q;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int i = g; i < count; i += DW_GROUPS) {
    const float4 v = *reinterpret_cast<const float4*>(p + static_cast<int64_t>(i) * K);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  s[g][q] = sum;
#pragma unroll
  for (int d = DW_GROUPS / 2; d >= 1; d >>= 1) {
    __syncthreads();
    if (g < d) {
      const float4 x = s[g][q], y = s[g + d][q];
      s[g][q] = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
  }
  if (g == 0) *reinterpret_cast<float4*>(dweight + blockIdx.x * (4 * DW_QUADS) + 4 * q) = s[0][q];
}

template <int WARPS, int VPT>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t stream) {
  constexpr int ROWS = norm_rows_per_cta<WARPS>();
  const unsigned grid = static_cast<unsigned>((a.rows + ROWS - 1) / ROWS);
  rmsnorm_rows_kernel<WARPS, VPT><<<grid, 32 * WARPS * ROWS, 0, stream>>>(a);
  return cudaGetLastError();
}

// With VPT granules a thread, in the first of WARPS, MORE... (ascending) that hold a row.
template <int VPT, int WARPS, int... MORE>
cudaError_t launch_rows_of(const NormArgs& a, cudaStream_t stream) {
  if constexpr (sizeof...(MORE) > 0)
    if (a.K > 512 * VPT * WARPS) return launch_rows_of<VPT, MORE...>(a, stream);
  return launch_rows<WARPS, VPT>(a, stream);
}

// Warps that take a row of K values in the backward pass: up to three vectors a thread, so
// that an SM holds several CTAs, each at another stage of a row (16384 x 5120: 99 us with
// 8 warps and three vectors, 118 with 16 and two; with four and half the warps 1000 x
// 4096 takes 12.8 us and with two 10.5, 16384 x 4096 84 and 82).
int back_warps(int64_t K) {
  int warps = 1;
  while (warps < 16 && K > 3 * 256 * warps) warps *= 2;
  return warps;
}
// Of the 228 KB of an SM; a CTA has 1 KB and its barriers and sums besides.
int back_shared(int warps) { return 228 * 1024 / (16 / warps) - 1024 - 512; }

template <int WARPS, int VECS, bool W32, bool KEEP>
cudaError_t launch_back_w(const NormBackArgs& a, int parts, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const int most = back_shared(WARPS), slot = a.K * (a.dh ? 6 : 4);
  const int stages = std::min(BACK_STAGES, most / slot);
  const auto kernel = rmsnorm_back_kernel<WARPS, VECS, W32, KEEP>;
  const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), most, &done);
  if (e != cudaSuccess) return e;
  kernel<<<parts, 32 * WARPS, stages * slot, stream>>>(a, stages);
  return cudaGetLastError();
}

template <int WARPS, int VECS, bool KEEP = true>
cudaError_t launch_back(const NormBackArgs& a, int parts, cudaStream_t stream) {
  return a.weight_f32 ? launch_back_w<WARPS, VECS, true, KEEP>(a, parts, stream)
                      : launch_back_w<WARPS, VECS, false, KEEP>(a, parts, stream);
}

// Two vectors a thread, or three.
template <int WARPS>
cudaError_t launch_back_few(const NormBackArgs& a, int parts, cudaStream_t stream) {
  return a.K <= 512 * WARPS ? launch_back<WARPS, 2>(a, parts, stream)
                            : launch_back<WARPS, 3>(a, parts, stream);
}

}  // namespace

cudaError_t launch_norm_rows(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const int granules = a.K / 16;
  // What counts in few rows is how long one takes, so a granule a thread (200 x 5120 2.8 us,
  // with two 3.1, with three 3.6), and in narrow ones.  Else two, in as many warps as the
  // row fills: 16384 x 5120 without a residual takes 47 us in five warps, 59 in eight; with
  // a residual 87 and 92.  Long runs without a residual, whose loads are half as many, have
  // three (9824 x 10240 59 us, with two 64), and narrow ones two (16384 x 1024 10.6 us, with
  // one 11.3; rstd alone 14.7 and 18.2 with the columns).  They have four where that is
  // four or eight warps with fewer idle lanes than three granules leave, above 7680 and
  // 15360 columns (rows of 134 M values, us with four and with three: 7424 columns 77.0, 72.6;
  // 7712 77.1, 80.1; 8192 72.9, 75.6; 10240, in five warps, 81.7, 77.0; 14336, in seven,
  // 81.7, 77.7; 15360 80.2, 75.8; 15392 81.9, 96.6; 16384 77.4, 91.0).
  const bool few = a.M <= 2 * num_sms, deep = !a.residual && a.M >= 32 * num_sms;
  if (deep && granules > 320 && granules <= 1024) {
    const int three = (granules + 95) / 96, four = (granules + 127) / 128;     // warps
    if (four % 4 == 0 && 128 * four < 96 * three) return launch_rows_of<4, 4, 8>(a, stream);
    return launch_rows_of<3, 4, 5, 6, 7, 8, 9, 10>(a, stream);
  }
  if (granules <= 32 || (granules <= 128 && !deep) || (granules <= 1024 && few))
    return launch_rows_of<1, 1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32>(a, stream);
  return launch_rows_of<2, 1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 32>(a, stream);
}

int norm_tile_rows() { return TILE_ROWS; }

cudaError_t launch_norm_both(const CUtensorMap& h, const CUtensorMap& q_col, const NormArgs& a,
                             uint8_t* s_col, uint32_t* dev_err, uint64_t timeout_ns, int num_sms,
                             cudaStream_t stream) {
  const int tiles_k = (a.K + MX_TILE_K - 1) / MX_TILE_K;
  const int64_t tiles = (static_cast<int64_t>(a.M) + TILE_ROWS - 1) / TILE_ROWS * tiles_k;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const cudaError_t e = launch_norm_rows(a, num_sms, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles));
  cfg.blockDim = dim3(TILE_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rmsnorm_cols_kernel, h, q_col, a, s_col, tiles_k,
                            num_sms * COL_CTAS / 2, dev_err, timeout_ns);
}

// As many CTAs as are resident at once, each of which takes as many rows as another.
int norm_back_parts(int64_t M, int64_t K, int num_sms) {
  const int warps = back_warps(K);
  const int64_t most = static_cast<int64_t>(num_sms) * (16 / warps);
  const int64_t turns = (M + most - 1) / most;
  return static_cast<int>((M + turns - 1) / turns);
}

cudaError_t launch_norm_back(const NormBackArgs& a, int parts, float* dweight, cudaStream_t stream) {
  cudaError_t e;
  switch (back_warps(a.K)) {
    case 1: e = launch_back_few<1>(a, parts, stream); break;
    case 2: e = launch_back_few<2>(a, parts, stream); break;
    case 4: e = launch_back_few<4>(a, parts, stream); break;
    case 8: e = launch_back_few<8>(a, parts, stream); break;
    default:
      e = a.K <= 12288   ? launch_back_few<16>(a, parts, stream)
          : a.K <= 16384 ? launch_back<16, 4>(a, parts, stream)
                         : launch_back<16, 8, false>(a, parts, stream);
  }
  if (e != cudaSuccess || !dweight) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.K / (4 * DW_QUADS)));
  cfg.blockDim = dim3(DW_QUADS * DW_GROUPS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rmsnorm_dweight_kernel, static_cast<const float*>(a.parts), parts,
                            a.K, dweight);
}

}  // namespace mxq
