// mx_tile.cuh -- MXFP8 of a 64 x 128 tile of fp32 values that the threads of a CTA hold
// in registers, LR x 8 values each (LR 4: 256 threads, LR 8: 128): codes and scales along
// the rows and along the columns.
//
// Warp w owns rows 2 LR w .. 2 LR w + 2 LR - 1 of the tile; lane (h, c) = (lane / 16,
// lane % 16) owns rows LR h .. LR h + LR - 1 and columns 8c .. 8c + 7 of those.  A row's
// block of 32 columns lies in four neighbouring lanes, a column's block of 32 rows in
// two lanes 16 apart of 16 / LR warps, which exchange their maxima through shared
// memory.  Rowwise codes leave as full 128-byte lines from registers; colwise codes are
// staged and leave by one bulk tensor store, 64 bytes a column; a row's four scale bytes
// leave as one store, and a column's two.
//
// 64 rows and not 128: four or five CTAs of 36 to 44 KiB an SM overlap one another's
// waits better than two of twice the size.
#pragma once

#include "mx_elements.cuh"
#include "mxq_internal.h"
#include "mxq_ptx.cuh"

namespace mxq {

constexpr int TILE_ROWS = 64;
constexpr int TILE_BLOCKS = TILE_ROWS / 32;                // colwise blocks
constexpr int TILE_CODES_BYTES = TILE_ROWS * MX_TILE_K;
template <int LR>
struct Tile {
  static_assert(LR == 4 || LR == 8, "rows a lane");
  static constexpr int WARPS = TILE_ROWS / (2 * LR);
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int BLOCK_WARPS = WARPS / TILE_BLOCKS;  // warps of a colwise block
  // [64][4] and [128][2] scale bytes, [WARPS][16][16 bytes] of maxima
  static constexpr int SCALES_BYTES = TILE_ROWS * 4 + MX_TILE_K * TILE_BLOCKS + WARPS * 256;
};

// Shared memory of one tile's way out, in bytes from its base.  `codes` is 1024-byte
// aligned (swizzled) and may lie elsewhere.
struct TileShared {
  uint32_t codes;      // [k % 8][k / 8][64 rows] colwise codes
  uint32_t row_scales;
  uint32_t col_scales;
  uint32_t maxima;
};

__device__ __forceinline__ TileShared tile_shared(uint32_t codes, uint32_t scales) {
  return {codes, scales, scales + TILE_ROWS * 4, scales + TILE_ROWS * 4 + MX_TILE_K * TILE_BLOCKS};
}

// Where a tile's results go.  Column 0 of the tile is column `col0` of the output
// (and of its scale rows), of which `width` columns exist from there on.
struct TileOut {
  int M;                 // rows of the matrix; row0 + its rows past M are not written
  int64_t pitch;         // columns of the whole output
  int row0, col0, width;
  uint8_t* q_row;
  uint8_t* s_row;
  uint8_t* s_col;
  const CUtensorMap* q_col;
  int qcol_x, qcol_y;    // the tile's place in the colwise code map (row, column / 8)
  int tiled;             // scales in 128 x 4 tiles
};

// Four scale bytes of each of `lines` rows at `src` to p + line * pitch, by THREADS threads
// t, a row each at least: parts of 32-byte sectors that neighbouring tiles complete, kept
// in L2 until they are whole.  `words`: all of them are aligned and four; else `n` exist,
// and neighbouring lanes have a row's bytes, so that they are one write of L2 as well
// (8192 x 14304: with a row's bytes by one lane 190 us forward and 193 backward, so 160
// and 177).
template <int THREADS>
__device__ __forceinline__ void store_row_scales(uint32_t src, int lines, uint8_t* p,
                                                 int64_t pitch, bool words, int n, int t) {
  if (words) {
    if (t < lines) stg32_hint(p + t * pitch, lds32(src + 4 * t), l2_policy_evict_last());
  } else {
#pragma unroll 1
    for (int k = t; k < 4 * lines; k += THREADS)
      if (k % 4 < n) stg8(p + k / 4 * pitch + k % 4, ld_shared_u8(src + k));
  }
}

// The tile's half of the 128 x 4 scale tiles of its rows and columns, one warp each.
// Where no tile has the other half (the last of an odd number) that is padding.
__device__ __forceinline__ void store_tile_row_scales(uint32_t src, int lane, uint8_t* tile,
                                                      int half, bool pad) {
  // Rows 32 g + lane at byte 16 lane + 4 g.
  uint8_t* p = tile + 16 * lane + 8 * half;
  stg64(p, lds32(src + 4 * lane), lds32(src + 4 * (lane + 32)));
  if (pad) stg64(p + 8, 0u, 0u);
}
__device__ __forceinline__ void store_tile_col_scales(uint32_t src, int lane, uint8_t* tile,
                                                      int half, bool pad) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t v = ld_shared_u16(src + 2 * (lane + 32 * g));
    uint8_t* p = tile + 16 * lane + 4 * g;
    if (pad) stg32(p, v);
    else stg16(p + 2 * half, v);
  }
}

// Scale exponents (f32_scale_exponent) of two magnitudes as 16-bit lanes.  Under the
// floor rule the exponent is in the upper half of each word.
__device__ __forceinline__ uint32_t exponent_pair(float a, float b, uint32_t ceil_f32) {
  if (ceil_f32 == 0u) return prmt(__float_as_uint(a), __float_as_uint(b), 0x7632) >> 7 & 0x00FF00FFu;
  return f32_scale_exponent(__float_as_uint(a), ceil_f32) |
         f32_scale_exponent(__float_as_uint(b), ceil_f32) << 16;
}

// 2^(127 - code) of the lower and the upper 16-bit lane of a pair of codes.
__device__ __forceinline__ float inv_scale_lo(uint32_t pair) {
  return __uint_as_float(0x7F000000u - (pair << 23));
}
__device__ __forceinline__ float inv_scale_hi(uint32_t pair) {
  return __uint_as_float(0x7F000000u - (pair << 7 & 0x7F800000u));
}

// The exponents of a lane's largest magnitudes: rows 2q, 2q + 1 and columns 2p, 2p + 1
// as 16-bit lanes.
template <int LR>
struct TileMaxima {
  uint32_t re[LR / 2], ce[4];
};

__device__ __forceinline__ float max8(const float (&r)[8]) {
  return fmax3(fmax3(fabsf(r[0]), fabsf(r[1]), fabsf(r[2])), fmax3(fabsf(r[3]), fabsf(r[4]), fabsf(r[5])),
               fmaxf(fabsf(r[6]), fabsf(r[7])));
}

template <int LR, bool ROW, bool COL>
__device__ __forceinline__ TileMaxima<LR> tile_maxima(const float (&y)[LR][8], uint32_t ceil_f32) {
  TileMaxima<LR> x;
  if constexpr (ROW) {
#pragma unroll
    for (int q = 0; q < LR / 2; ++q)
      x.re[q] = exponent_pair(max8(y[2 * q]), max8(y[2 * q + 1]), ceil_f32);
  }
  if constexpr (COL) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float m[2];
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const int j = 2 * p + d;
        m[d] = fmaxf(fmax3(fabsf(y[0][j]), fabsf(y[1][j]), fabsf(y[2][j])), fabsf(y[3][j]));
        if constexpr (LR == 8)
          m[d] = fmax3(fmax3(fabsf(y[4][j]), fabsf(y[5][j]), fabsf(y[6][j])), fabsf(y[7][j]), m[d]);
      }
      x.ce[p] = exponent_pair(m[0], m[1], ceil_f32);
    }
  }
  return x;
}

// Before a barrier: the columns' exponents over the warp's rows, published for the
// other warps of the block.
template <int LR>
__device__ __forceinline__ void publish_columns(TileMaxima<LR>& x, uint32_t maxima) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int p = 0; p < 4; ++p) x.ce[p] = vmax_u16x2(x.ce[p], __shfl_xor_sync(0xFFFFFFFFu, x.ce[p], 16));
  if (lane < 16) sts128(maxima + (warp * 16 + lane) * 16, x.ce[0], x.ce[1], x.ce[2], x.ce[3]);
}

// After that barrier: rowwise codes to memory, colwise codes and all scales to the
// staging, which is free by then.
template <int LR, bool ROW, bool COL>
__device__ __forceinline__ void emit_tile(const float (&y)[LR][8], const TileMaxima<LR>& x,
                                          const TileShared& sh, const TileOut& o) {
  using T = Tile<LR>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = lane >> 4, c = lane & 15;
  const int rl = 2 * LR * warp + LR * h;
  if constexpr (ROW) {
    uint32_t rc[LR / 2];
#pragma unroll
    for (int q = 0; q < LR / 2; ++q) {
      uint32_t e = x.re[q];
      e = vmax_u16x2(e, __shfl_xor_sync(0xFFFFFFFFu, e, 1));
      e = vmax_u16x2(e, __shfl_xor_sync(0xFFFFFFFFu, e, 2));
      rc[q] = e8m0_pair(e);
    }
    const bool ok = o.row0 + rl < o.M && 8 * c < o.width;
    uint8_t* q = o.q_row + static_cast<int64_t>(o.row0 + rl) * o.pitch + o.col0 + 8 * c;
#pragma unroll
    for (int i = 0; i < LR; ++i) {
      const float inv = i & 1 ? inv_scale_hi(rc[i >> 1]) : inv_scale_lo(rc[i >> 1]);
      uint32_t w[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 v = mul_f32x2(make_float2(y[i][2 * p], y[i][2 * p + 1]), f2(inv));
        w[p] = cvt_e4m3x2(v.x, v.y);
      }
      if (ok) stg64_cs(q + i * o.pitch, w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
    // The lane stages rows c % 4 (and c % 4 + 4) of its own, block c / 4.
    const uint32_t at = sh.row_scales + (rl + (c & 3)) * 4 + (c >> 2);
    sts8(at, half16(c & 2 ? rc[1] : rc[0], c & 1) & 0xFFu);
    if constexpr (LR == 8) sts8(at + 16, half16(c & 2 ? rc[3] : rc[2], c & 1) & 0xFFu);
  }
  if constexpr (COL) {
    // The other warps of the 32 rows.
    uint32_t m[4] = {x.ce[0], x.ce[1], x.ce[2], x.ce[3]};
#pragma unroll
    for (int d = 1; d < T::BLOCK_WARPS; ++d) {
      const uint4 v = lds128(sh.maxima + ((warp ^ d) * 16 + c) * 16);
      m[0] = vmax_u16x2(m[0], v.x);
      m[1] = vmax_u16x2(m[1], v.y);
      m[2] = vmax_u16x2(m[2], v.z);
      m[3] = vmax_u16x2(m[3], v.w);
    }
    // [k % 8][k / 8][64 rows], the 16-byte chunk index xor-ed with (k / 16) % 4 (the
    // 64-byte swizzle of the store's tensor map).
    const uint32_t at = sh.codes + c * TILE_ROWS + (((rl >> 4) ^ ((c >> 1) & 3)) << 4) + (rl & 15);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t cc = m[p] = e8m0_pair(m[p]);
      const float2 iv = make_float2(inv_scale_lo(cc), inv_scale_hi(cc));
      uint32_t we[LR / 2], wo[LR / 2];
#pragma unroll
      for (int i = 0; i < LR; i += 2) {
        const float2 r0 = mul_f32x2(make_float2(y[i][2 * p], y[i][2 * p + 1]), iv);
        const float2 r1 = mul_f32x2(make_float2(y[i + 1][2 * p], y[i + 1][2 * p + 1]), iv);
        we[i / 2] = cvt_e4m3x2(r0.x, r1.x);
        wo[i / 2] = cvt_e4m3x2(r0.y, r1.y);
      }
      const uint32_t even = at + (2 * p) * 16 * TILE_ROWS, odd = even + 16 * TILE_ROWS;
      if constexpr (LR == 8) {
        sts64(even, we[0] | (we[1] << 16), we[2] | (we[3] << 16));
        sts64(odd, wo[0] | (wo[1] << 16), wo[2] | (wo[3] << 16));
      } else {
        sts32(even, we[0] | (we[1] << 16));
        sts32(odd, wo[0] | (wo[1] << 16));
      }
    }
    // One warp of a block writes its scales, h = 0 columns 8c .. 8c + 3 and h = 1 the
    // others: [128 columns][2].
    if (warp % T::BLOCK_WARPS == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sts8(sh.col_scales + (c * 8 + 4 * h + j) * TILE_BLOCKS + warp / T::BLOCK_WARPS,
             half16(h ? m[2 + (j >> 1)] : m[j >> 1], j & 1) & 0xFFu);
    }
    fence_proxy_async_smem();
  }
}

// After another barrier: the colwise codes' bulk store, which thread 0 waits for
// (bulk_wait_read) before the CTA ends, and the scales.
template <int LR, bool ROW, bool COL>
__device__ __forceinline__ void finish_tile(const TileShared& sh, const TileOut& o) {
  using T = Tile<LR>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (COL && tid == 0) {
    tma_store_3d(o.q_col, sh.codes, o.qcol_x, o.qcol_y, 0);
    bulk_commit();
  }
  const int64_t nkb = o.pitch / 32;
  const int nmb = o.M / 32;
  if (o.tiled) {
    const int half = o.row0 >> 6 & 1;
    const bool pad = half == 0 && o.row0 + TILE_ROWS >= o.M;
    if (ROW && warp == 1)
      store_tile_row_scales(sh.row_scales, lane,
                            o.s_row + ((o.row0 >> 7) * ((nkb + 3) / 4) + (o.col0 >> 7)) * 512, half, pad);
    if (COL && warp == 2)
      store_tile_col_scales(sh.col_scales, lane,
                            o.s_col + (static_cast<int64_t>(o.col0 >> 7) * ((nmb + 3) / 4) +
                                       (o.row0 >> 7)) * 512, half, pad);
  } else {
    // Threads 0 .. 127 the columns', the last 64 the rows'.
    if (COL && tid < o.width) {
      // Two bytes a column, one where the matrix ends.
      uint8_t* p = o.s_col + static_cast<int64_t>(o.col0 + tid) * nmb + o.row0 / 32;
      const uint32_t v = ld_shared_u16(sh.col_scales + 2 * tid);
      if ((nmb & 1) == 0) {
        stg16_hint(p, v, l2_policy_evict_last());
      } else {
        stg8(p, v & 0xFFu);
        if (o.row0 / 32 + 1 < nmb) stg8(p + 1, v >> 8);
      }
    }
    if constexpr (ROW)
      store_row_scales<T::THREADS>(sh.row_scales, min(TILE_ROWS, o.M - o.row0),
                                   o.s_row + o.row0 * nkb + o.col0 / 32, nkb,
                                   o.width == MX_TILE_K && ((nkb | o.col0 / 32) & 3) == 0,
                                   o.width / 32, (tid + TILE_ROWS) % T::THREADS);
  }
}

// All of it, by every thread of the CTA.  The staging is free by the first barrier,
// which may be what frees it.
template <int LR, bool ROW, bool COL>
__device__ __forceinline__ void quantize_tile(const float (&y)[LR][8], const TileShared& sh,
                                              const TileOut& o, uint32_t ceil_f32) {
  TileMaxima<LR> x = tile_maxima<LR, ROW, COL>(y, ceil_f32);
  if constexpr (COL) publish_columns(x, sh.maxima);
  __syncthreads();
  emit_tile<LR, ROW, COL>(y, x, sh, o);
  __syncthreads();
  finish_tile<LR, ROW, COL>(sh, o);
}

}  // namespace mxq
