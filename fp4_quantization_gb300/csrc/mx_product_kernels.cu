// mx_product_kernels.cu -- products grouped by expert on MXFP8 operands.
//
// out_g = A_g B_g^T with E4M3 codes and one E8M0 scale per 32 values of the
// contraction axis: sum_k a[m, k] 2^(sa[m, k / 32] - 127) b[n, k]
// 2^(sb[n, k / 32] - 127).  The tensor cores apply both scales
// (tcgen05.mma kind::mxf8f6f4, one scale per 32 values of K) and accumulate
// in fp32 in tensor memory.
#include "mxq_products.h"

#include "mxq_tc_ptx.cuh"

namespace mxq {
namespace {

constexpr int TILE_M = 128;           // output rows of a tile: the instruction's M
constexpr int STEP_K = 128;           // contraction bytes of one pipeline stage: a swizzle row
constexpr int CHUNK = 4;              // stages that share one set of scale tiles (16 bytes a row)
constexpr int THREADS = 320;          // 4 epilogue, 4 scale, 1 copy, 1 issuing warp
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SCALE_COL = 480;   // first tensor-memory column of the scales

template <int BN>
struct Shape {
  static constexpr int A_BYTES = TILE_M * STEP_K;
  static constexpr int B_BYTES = BN * STEP_K;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 4 : 5;
  static constexpr int B_TILES = (BN + 127) / 128;                  // scale tiles of B a stage
  static constexpr int SCALE_BYTES = CHUNK * 512 * (1 + B_TILES);   // one scale chunk
  static constexpr int SCALE_CHUNKS = 2;
  // Column of accumulator s.  Two 256-column accumulators share 32 columns.
  static constexpr uint32_t acc_col(uint32_t s) { return s * (BN == 256 ? 224 : BN); }
  static constexpr int TABLE_BYTES = 2 * (GROUPS_MAX + 1) * 4;
  static constexpr int BARRIERS = 2 * STAGES + 2 * SCALE_CHUNKS + 4 + 1;
  static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + SCALE_CHUNKS * SCALE_BYTES +
                              TABLE_BYTES + BARRIERS * 8 + 64;
};

// Where a tile lies: its group, its first row and column in the group's
// output, and the group's rows and contraction range.
struct Tile {
  int g, m0, n0;
  int rows;         // rows of the group's output
  int first, depth; // contraction range (wgrad: first row of the group; forward: 0)
};

// Walks the tiles of this CTA in order.  Inside a group the row tiles of a
// band of 16 run fastest, so a wave's tiles share their rows and read each
// column tile's codes from memory once a band.
template <bool WGRAD>
struct Walk {
  const int* off;
  const int* start;     // first tile of each group, and the total
  int groups, tiles_n;
  int t, g;

  template <int BN>
  __device__ __forceinline__ bool next(const GroupedArgs& a, Tile& tile) {
    if (t >= start[groups]) return false;
    while (t >= start[g + 1]) ++g;
    const int lo = off[g], rows_g = off[g + 1] - lo;
    tile.g = g;
    tile.rows = WGRAD ? a.a_rows : rows_g;
    tile.first = WGRAD ? lo : 0;
    tile.depth = WGRAD ? rows_g : a.depth;
    constexpr int BAND = 16;
    const int tiles_m = (tile.rows + TILE_M - 1) / TILE_M;
    int i = t - start[g];
    const int band = i / (BAND * tiles_n);
    i -= band * BAND * tiles_n;
    const int height = min(BAND, tiles_m - band * BAND);
    tile.m0 = (band * BAND + i % height) * TILE_M;
    tile.n0 = i / height * BN;
    t += gridDim.x;
    return true;
  }
};

// 16 scale bytes from p on, of a row with `valid` bytes left, in a matrix that
// ends at `end`.  Rows of scales start at any byte, so the bytes come from the
// one or two 16-byte blocks around them; what follows the row's bytes is read
// by no instruction.  Blocks that the matrix's end cuts are read by bytes.
__device__ __forceinline__ uint4 load_scales(const uint8_t* p, int valid, const uint8_t* end) {
  if (valid <= 0) return make_uint4(0, 0, 0, 0);
  const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15;
  const uint8_t* block = p - shift;
  const bool two = shift + min(valid, 16) > 16;
  if (block + (two ? 32 : 16) > end) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < valid) w[i / 4] |= static_cast<uint32_t>(__ldg(p + i)) << (8 * (i % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  const uint4 lo = __ldg(reinterpret_cast<const uint4*>(block));
  if (shift == 0) return lo;
  const uint4 hi = two ? __ldg(reinterpret_cast<const uint4*>(block) + 1) : lo;
  uint32_t w[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z};
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 2];
    w[5] = hi.w;
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = w[i + 1];
    w[4] = w[5];
  }
  const uint32_t bits = 8 * (shift & 3);
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// Writes row r's scales of the four stages of a chunk into their tiles.
__device__ __forceinline__ void store_scales(uint32_t tiles, int r, uint4 v) {
  const uint32_t at = tiles + (r % 32) * 16 + (r / 32) * 4;
  sts32(at, v.x);
  sts32(at + 512, v.y);
  sts32(at + 1024, v.z);
  sts32(at + 1536, v.w);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// One lane's 32 consecutive columns of an output row; `cols` of them exist.
__device__ __forceinline__ void store_row(const GroupedArgs& a, int64_t row, int col, int cols,
                                          const uint32_t (&v)[32]) {
  if (a.out_f32) {
    float* p = static_cast<float*>(a.out) + row * a.ldo + col;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      if (a.out_vec && i + 4 <= cols) {
        stg128(p + i, v[i], v[i + 1], v[i + 2], v[i + 3]);
      } else {
#pragma unroll
        for (int j = i; j < i + 4; ++j)
          if (j < cols) p[j] = __uint_as_float(v[j]);
      }
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(a.out) + row * a.ldo + col;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack_bf16(__uint_as_float(v[i + 2 * j]), __uint_as_float(v[i + 2 * j + 1]));
      if (a.out_vec && i + 8 <= cols) {
        stg128(p + i, w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i + j < cols) p[i + j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
      }
    }
  }
}

template <int BN, bool WGRAD>
__global__ void __launch_bounds__(THREADS, 1)
mx_grouped_kernel(const __grid_constant__ GroupedMaps maps, const GroupedArgs a) {
  using S = Shape<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_up_shared<1024>(smem_raw);
  const uint32_t stages = smem_addr(smem);
  const uint32_t scales = stages + S::STAGES * S::STAGE_BYTES;
  int* off = reinterpret_cast<int*>(smem + S::STAGES * S::STAGE_BYTES +
                                    S::SCALE_CHUNKS * S::SCALE_BYTES);
  int* start = off + GROUPS_MAX + 1;
  const uint32_t bars = smem_addr(start + GROUPS_MAX + 1);   // 8-byte aligned: 2 (MAX + 1) words
  const uint32_t full = bars, empty = full + 8 * S::STAGES;
  const uint32_t sc_full = empty + 8 * S::STAGES, sc_empty = sc_full + 8 * S::SCALE_CHUNKS;
  const uint32_t acc_full = sc_empty + 8 * S::SCALE_CHUNKS, acc_empty = acc_full + 16;
  const uint32_t drain = acc_empty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(start + GROUPS_MAX + 1) + 2 * S::BARRIERS;

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int tiles_n = (a.b_rows + BN - 1) / BN;

  if (tid == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < S::SCALE_CHUNKS; ++i) {
      mbar_init(sc_full + 8 * i, 128);
      mbar_init(sc_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 128);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(smem_addr(tmem_slot), TMEM_COLS);

  // Offsets, checked, and the groups' first tiles (each warp's share scanned
  // by shuffles, 32 groups a step).
  bool bad = false;
  for (int i = tid; i <= a.groups; i += THREADS) {
    const int v = a.offsets[i];
    const int before = i > 0 ? a.offsets[i - 1] : 0;
    bad |= v < before || v > a.limit || (WGRAD && v % 32 != 0);
    off[i] = v;
  }
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    int total = 0;
    for (int i = 0; i < a.groups; i += 32) {
      int n = 0;
      if (!bad && i + lane < a.groups) {
        const int rows = WGRAD ? a.a_rows : off[i + lane + 1] - off[i + lane];
        n = (rows + TILE_M - 1) / TILE_M * tiles_n;
      }
      int sum = n;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int up = __shfl_up_sync(~0u, sum, d);
        if (lane >= d) sum += up;
      }
      if (i + lane < a.groups) start[i + lane] = total + sum - n;
      total += __shfl_sync(~0u, sum, 31);
    }
    if (lane == 0) start[a.groups] = total;
    if (bad && lane == 0 && blockIdx.x == 0 && a.dev_err) atomicOr(a.dev_err, MXQ_DEVERR_OFFSETS);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  Walk<WGRAD> walk{off, start, a.groups, tiles_n, static_cast<int>(blockIdx.x), 0};
  Tile tile;
  bool ok = true;

  if (warp == 8) {
    // ---- copies: one stage of A and B codes at a time ----
    if (lane == 0) {
      uint32_t it = 0;
      while (ok && walk.template next<BN>(a, tile)) {
        const int steps = (tile.depth + STEP_K - 1) / STEP_K;
        const int ay = WGRAD ? tile.m0 : off[tile.g] + tile.m0;
        const int bz = WGRAD ? 0 : tile.g;
        for (int k = 0; k < steps; ++k, ++it) {
          const uint32_t s = it % S::STAGES;
          if (it >= S::STAGES &&
              !mbar_wait_bounded(empty + 8 * s, (it / S::STAGES - 1) & 1, a.timeout_ns)) {
            ok = false;
            break;
          }
          const uint32_t dst = stages + s * S::STAGE_BYTES, bar = full + 8 * s;
          mbar_arrive_expect_tx(bar, S::STAGE_BYTES);
          const int x = tile.first + k * STEP_K;
          tma_load_2d(dst, &maps.a, x, ay, bar);
          tma_load_3d(dst + S::A_BYTES, &maps.b, x, tile.n0, bz, bar);
        }
      }
      // After a wait that ran out, the copies in flight still land.
      if (!ok)
        for (uint32_t i = it > S::STAGES ? it - S::STAGES : 0; i < it; ++i)
          mbar_wait_bounded(full + 8 * (i % S::STAGES), (i / S::STAGES) & 1, a.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---- tensor-core instructions ----
    if (lane == 0) {
      uint32_t it = 0, chunk = 0, acc = 0;
      while (ok && walk.template next<BN>(a, tile)) {
        const int steps = (tile.depth + STEP_K - 1) / STEP_K;
        if (steps == 0) continue;
        // The accumulator's columns are free: for 256 columns, the shared 32
        // of the tile before (whose readers have then finished the tile
        // before that); otherwise, all of the tile two before.
        const uint32_t lag = BN == 256 ? 1 : 2;
        if (acc >= lag && !mbar_wait_bounded(acc_empty + 8 * ((acc - lag) % 2),
                                             ((acc - lag) / 2) & 1, a.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem + S::acc_col(acc % 2);
        for (int k = 0; ok && k < steps; ++k, ++it) {
          const uint32_t c = chunk % S::SCALE_CHUNKS, s = it % S::STAGES;
          if (k % CHUNK == 0 &&
              !mbar_wait_bounded(sc_full + 8 * c, (chunk / S::SCALE_CHUNKS) & 1, a.timeout_ns))
            ok = false;
          if (!ok || !mbar_wait_bounded(full + 8 * s, (it / S::STAGES) & 1, a.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          // Scales of this stage: A's tile, then B's, in alternating columns.
          const uint32_t sc = scales + c * S::SCALE_BYTES + (k % CHUNK) * 512;
          const uint32_t ts = tmem + SCALE_COL + (k % 2) * 16;
          tc_copy_scales(ts, scale_desc(sc));
#pragma unroll
          for (int b = 0; b < S::B_TILES; ++b)
            tc_copy_scales(ts + 4 + 4 * b, scale_desc(sc + (1 + b) * CHUNK * 512));
          const uint64_t da = operand_desc(stages + s * S::STAGE_BYTES);
          const uint64_t db = operand_desc(stages + s * S::STAGE_BYTES + S::A_BYTES);
          const int left = (tile.depth - k * STEP_K) / 32;
#pragma unroll
          for (int j = 0; j < STEP_K / 32; ++j)
            if (j < left)
              tc_mma_mxf8(d, da + 2 * j, db + 2 * j, mxf8_idesc(TILE_M, BN, j), ts, ts + 4,
                          k > 0 || j > 0);
          tc_commit(empty + 8 * s);
          if (k % CHUNK == CHUNK - 1 || k == steps - 1) {
            tc_commit(sc_empty + 8 * c);
            ++chunk;
          }
        }
        if (ok) tc_commit(acc_full + 8 * (acc % 2));
        ++acc;
      }
      // Nothing of this thread's is in flight when the memory is given back.
      if (!ok) {
        tc_commit(drain);
        mbar_wait_bounded(drain, 0, a.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---- scales: thread r takes rows r of A and r, r + 128 of B ----
    const int r = tid - 128;
    const uint8_t* a_end = a.a_s + static_cast<int64_t>(WGRAD ? a.a_rows : a.limit) * a.s_ld;
    const uint8_t* b_end = a.b_s + (WGRAD ? 1 : a.groups) * static_cast<int64_t>(a.b_rows) * a.s_ld;
    uint32_t chunk = 0;
    while (ok && walk.template next<BN>(a, tile)) {
      const int steps = (tile.depth + STEP_K - 1) / STEP_K;
      const int blocks = tile.depth / 32;
      const int64_t arow = (WGRAD ? 0 : off[tile.g]) + tile.m0 + r;
      const bool ahas = tile.m0 + r < tile.rows;
      const uint8_t* ap = a.a_s + arow * a.s_ld + tile.first / 32;
      const uint8_t* bp = a.b_s +
          ((WGRAD ? 0 : static_cast<int64_t>(tile.g) * a.b_rows) + tile.n0 + r) * a.s_ld +
          tile.first / 32;
      for (int k = 0; k < steps; k += CHUNK, ++chunk) {
        const uint32_t c = chunk % S::SCALE_CHUNKS;
        const int at = k * (STEP_K / 32), valid = blocks - at;
        const uint4 va = load_scales(ap + at, ahas ? valid : 0, a_end);
        uint4 vb[S::B_TILES];
#pragma unroll
        for (int b = 0; b < S::B_TILES; ++b)
          vb[b] = load_scales(bp + b * 128 * a.s_ld + at,
                              tile.n0 + r + b * 128 < a.b_rows && r + b * 128 < BN ? valid : 0,
                              b_end);
        if (chunk >= S::SCALE_CHUNKS &&
            !mbar_wait_bounded(sc_empty + 8 * c, (chunk / S::SCALE_CHUNKS - 1) & 1, a.timeout_ns)) {
          ok = false;
          break;
        }
        const uint32_t dst = scales + c * S::SCALE_BYTES;
        store_scales(dst, r, va);
#pragma unroll
        for (int b = 0; b < S::B_TILES; ++b) store_scales(dst + (1 + b) * CHUNK * 512, r, vb[b]);
        fence_proxy_async_smem();
        mbar_arrive(sc_full + 8 * c);
      }
    }
  } else {
    // ---- epilogue: warp w reads lanes 32 w .. 32 w + 31, a row each ----
    uint32_t acc = 0;
    while (ok && walk.template next<BN>(a, tile)) {
      const int row = tile.m0 + tid;
      const bool live = row < tile.rows;
      const int64_t out_row = WGRAD ? static_cast<int64_t>(tile.g) * a.a_rows + row
                                    : static_cast<int64_t>(off[tile.g]) + row;
      uint32_t v[32];
      if (tile.depth == 0) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0;
        for (int j = 0; j < BN; j += 32)
          if (live) store_row(a, out_row, tile.n0 + j, a.b_rows - tile.n0 - j, v);
        continue;
      }
      const uint32_t s = acc % 2;
      if (!mbar_wait_bounded(acc_full + 8 * s, (acc / 2) & 1, a.timeout_ns)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t base = tmem + S::acc_col(s) + (static_cast<uint32_t>(warp) << 21);
      for (int i = 0; i < BN / 32; ++i) {
        // Accumulator 0 shares its last 32 columns with the next tile's
        // first 32: they are read first.
        const int j = 32 * (BN == 256 && s == 0 ? BN / 32 - 1 - i : i);
        tmem_load_x32(base + j, v);
        tmem_wait_load();
        if (i == (BN == 256 ? 0 : BN / 32 - 1)) {
          tc_fence_before_sync();
          mbar_arrive(acc_empty + 8 * s);
        }
        if (live) store_row(a, out_row, tile.n0 + j, a.b_rows - tile.n0 - j, v);
      }
      ++acc;
    }
  }

  if (!ok && a.dev_err) atomicOr(a.dev_err, MXQ_DEVERR_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 9) tmem_dealloc(tmem, TMEM_COLS);
}

template <int BN, bool WGRAD>
cudaError_t launch(const GroupedMaps& maps, const GroupedArgs& a, int num_sms,
                   cudaStream_t stream) {
  auto kernel = mx_grouped_kernel<BN, WGRAD>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Shape<BN>::SMEM);
  if (e != cudaSuccess) return e;
  // At most this many tiles, whatever the offsets are.
  const int64_t tiles_n = (a.b_rows + BN - 1) / BN;
  const int64_t tiles_m =
      WGRAD ? static_cast<int64_t>(a.groups) * ((a.a_rows + TILE_M - 1) / TILE_M)
            : a.limit / TILE_M + (a.groups < a.limit ? a.groups : a.limit);
  const int64_t tiles = tiles_m * tiles_n;
  const int grid = static_cast<int>(tiles < num_sms ? tiles : num_sms);
  kernel<<<grid, THREADS, Shape<BN>::SMEM, stream>>>(maps, a);
  return cudaGetLastError();
}

}  // namespace

int grouped_tile_cols(int64_t rows, int64_t cols, int groups, int num_sms) {
  const int64_t tiles_m = rows / TILE_M + groups;
  return tiles_m * ((cols + 255) / 256) >= 2 * num_sms ? 256 : 128;
}

cudaError_t launch_grouped(const GroupedMaps& maps, const GroupedArgs& a, bool wgrad,
                           int tile_cols, int num_sms, cudaStream_t stream) {
  if (wgrad)
    return tile_cols == 256 ? launch<256, true>(maps, a, num_sms, stream)
                            : launch<128, true>(maps, a, num_sms, stream);
  return tile_cols == 256 ? launch<256, false>(maps, a, num_sms, stream)
                          : launch<128, false>(maps, a, num_sms, stream);
}

}  // namespace mxq
