// mx_product_kernels.cu -- products grouped by expert on MXFP8 operands.
//
// out_g = A_g B_g^T with E4M3 codes and one E8M0 scale per 32 values of the
// contraction axis: sum_k a[m, k] 2^(sa[m, k / 32] - 127) b[n, k]
// 2^(sb[n, k / 32] - 127).  The tensor cores apply both scales
// (tcgen05.mma kind::mxf8f6f4, one scale per 32 values of K) and accumulate
// in fp32 in tensor memory.
//
// Large calls are bound by the board's power and then by the tensor pipe (8192
// rows over 8 experts, 4096 x 8192: 187 us, 2.9 PFLOP/s, for the first hundred
// calls, 191-205 on and on, 166 on zero codes, at which the clock stays up; 16384
// rows, 14336 x 4096: 632-647, 672-705 and 546 us), calls with
// few rows an expert by reading the weights (36 rows over 41 experts, 5866 x
// 1344: 33 us, 5.9 TB/s), weight gradients of short groups by writing them (64
// experts x 1408 x 2048 fp32: 132 us, 5.8 TB/s).
#include <type_traits>

#include "mxq_products.h"

#include "mxq_tc_ptx.cuh"

namespace mxq {
namespace {

constexpr int ROWS = 128;             // output rows of a CTA's tile
constexpr int STEP_K = 128;           // contraction bytes of one pipeline stage: a swizzle row
// Stages whose scales are fetched together: 64 bytes a row, by four threads in
// one request.  The scales are 3% of the bytes, but fetched 16 bytes at a time
// they were 27% of the requests to L2, and the codes' copies waited for them.
constexpr int WINDOW = 16;
constexpr int THREADS = 320;          // 4 epilogue, 4 scale, 1 copy, 1 issuing warp
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SCALE_COL = 480;   // first tensor-memory column of the scales
// Rows of a group on average up to which they are the narrow operand (FEW): 0.9
// rows of 41 experts x 5866 x 1344 34 us so and 49 as 128-row operands, 64 rows
// of 64 experts x 1408 x 2048 60 us so and 43.
constexpr int FEW_ROWS = 32;
// Contraction values after which an fp32 output's sum is taken out of tensor
// memory and added in fp32: the tensor cores cut their sums off towards zero
// instead of rounding them, which on random operands leaves errors of 7.4e-8 of
// the result's norm after 1056 values, 1.3e-7 after 2048, 2.8e-7 after 4096 and
// 6.6e-7 after 8192 (fp32 additions: 4.6e-8, 6.3e-8, 9.4e-8, 1.4e-7).  A range more
// writes and adds the whole output once more: with 4096 here 4096 rows over 8
// experts, 4096 x 8192, take 161 us instead of 114, 1772 over 7, 3361 x 4384, whose
// rows are not aligned, 182 instead of 47.
constexpr int SEGMENT = 8192;
// Ranges of the contraction that the CTAs of a cluster take at most, and the
// stages of one at least (16 rows x 4096 x 14336: 32.4 us whole, 20.9 in halves,
// 15.7 in quarters, 15.8 in eighths; 8 x 2048 x 2048, 16 stages, 8.1, 7.2, 6.2).
// Adding them up takes as long as some four stages: 8 are not divided (128 x 512 x
// 1024 6.9 us whole, 8.6 in halves).
constexpr int SPLIT_MAX = 4;
constexpr int SPLIT_STEPS = 4;

// What the two operands and the output tile are.
//  FORWARD: A the rows of x of a group, B its expert's weight.
//  FEW:     A the weight, B the rows of x: the tile is the output's transpose.
//           Few rows fill a fraction of a 128-row operand, and its other rows
//           would be half of all that is copied; here they are the narrow one.
//  WGRAD:   A the gradient, B x, both along the group's rows.
enum Kind { FORWARD, FEW, WGRAD };

// A tile of ROWS * CTAS rows and BN columns, worked on by one CTA or a pair.
template <int CTAS, int BN>
struct Shape {
  static constexpr int A_BYTES = ROWS * STEP_K;
  static constexpr int B_ROWS = BN / CTAS;                          // of each CTA
  static constexpr int STAGE_BYTES = A_BYTES + B_ROWS * STEP_K;
  static constexpr int STAGES = STAGE_BYTES > 40 * 1024 ? 4 : BN >= 128 ? 5 : 8;
  static constexpr int B_TILES = (BN + 127) / 128;                  // scale tiles of B a stage
  // Stages whose scales share a place in shared memory: the fewer, the more is
  // left for codes in flight, which bound large calls (a pair's fifth stage: gemm
  // 16384 x 14336 x 4096 over 8 experts 686 -> 660 us).
  static constexpr int CHUNK = STAGE_BYTES > 40 * 1024 ? 4 : 8;
  static constexpr int SCALE_BYTES = CHUNK * 512 * (1 + B_TILES);   // one scale chunk
  static constexpr int SCALE_CHUNKS = 2;
  // Patches of 32 rows x 128 bytes that the epilogue's four warps stage: two
  // each, one filled while the other leaves (one where shared memory is short).
  static constexpr int PATCHES = BN < 128 ? 0 : STAGE_BYTES > 40 * 1024 ? 1 : 2;
  static constexpr int OUT_BYTES = 4 * PATCHES * 4096;
  // Column of accumulator s.  Two 256-column accumulators share 32 columns.
  static constexpr uint32_t acc_col(uint32_t s) { return s * (BN == 256 ? 224 : BN); }
  static constexpr int TABLE_BYTES = 2 * (GROUPS_MAX + 1) * 4;
  static constexpr int BARRIERS = 2 * STAGES + 2 * SCALE_CHUNKS + 4 + 1;
  static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + SCALE_CHUNKS * SCALE_BYTES +
                              OUT_BYTES + TABLE_BYTES + BARRIERS * 8 + 16;
};

// Where a tile lies: its group, its first row and column in the group's
// product, that product's rows and columns, and the tile's contraction range.
struct Tile {
  int g, m0, n0;
  int rows, cols;
  int first, end;   // contraction range
  bool add;         // to what an earlier range of the tile has written
  int ay, az;       // the product's first row in A: row ay of matrix az,
  int by, bz;       // and its first column in B

  // Stages start on whole swizzle rows, so that their scales are whole words
  // and, where scale rows are multiples of 16 bytes, chunks whole 64-byte
  // pieces of them; the blocks of 32 before `first` are skipped.
  __device__ __forceinline__ int step0() const { return first / STEP_K; }
  __device__ __forceinline__ int step1() const {
    return first < end ? (end + STEP_K - 1) / STEP_K : step0();
  }
};

// Walks the tiles of this CTA (or pair) in order.  Inside a group the row
// tiles of a band of 2048 rows run fastest, so a wave's tiles share their rows
// and each column tile's codes come from memory once a band; with few rows of
// x, all of them beside each weight tile.  With SPLIT the CTAs of a cluster take
// a range of the contraction each, of one tile.
template <int CTAS, int BN, int KIND, bool SPLIT = false>
struct Walk {
  const int* off;
  const int* start;     // first tile of each group, and the total
  int groups;
  int t, g, done;       // done: where tile t's next contraction range starts, or 0

  __device__ __forceinline__ bool next(const GroupedArgs& a, Tile& tile) {
    if (t >= start[groups]) return false;
    while (t >= start[g + 1]) ++g;
    const int lo = off[g], rows_g = off[g + 1] - lo;
    tile.g = g;
    tile.rows = KIND == FORWARD ? rows_g : a.a_rows;
    tile.cols = KIND == FEW ? rows_g : a.b_rows;
    tile.ay = KIND == FORWARD ? lo : 0;
    tile.az = KIND == FEW ? g : 0;
    tile.by = KIND == FEW ? lo : 0;
    tile.bz = KIND == FORWARD ? g : 0;
    const int from = KIND == WGRAD ? lo : 0, to = KIND == WGRAD ? lo + rows_g : a.depth;
    tile.add = done > 0;
    tile.first = tile.add ? done : from;
    tile.end = a.out_f32 ? min(to, (tile.first / STEP_K + SEGMENT / STEP_K) * STEP_K) : to;
    if constexpr (SPLIT) {
      // Whole stages, so that no two CTAs copy the same one.
      const int step0 = from / STEP_K, steps = (to + STEP_K - 1) / STEP_K - step0;
      const int each = (steps + a.split - 1) / a.split;
      const int at = step0 + min(static_cast<int>(cluster_rank()) * each, steps);
      tile.first = min(max(at * STEP_K, from), to);
      tile.end = min(min(at + each, step0 + steps) * STEP_K, to);
      tile.add = false;
    }
    const int tiles_n = (tile.cols + BN - 1) / BN;
    int i = t - start[g];
    if constexpr (KIND == FEW) {
      tile.m0 = i / tiles_n * (ROWS * CTAS);
      tile.n0 = i % tiles_n * BN;
    } else {
      constexpr int BAND = 2048 / (ROWS * CTAS);
      const int tiles_m = (tile.rows + ROWS * CTAS - 1) / (ROWS * CTAS);
      const int band = i / (BAND * tiles_n);
      i -= band * BAND * tiles_n;
      const int height = min(BAND, tiles_m - band * BAND);
      tile.m0 = (band * BAND + i % height) * (ROWS * CTAS);
      tile.n0 = i / height * BN;
    }
    done = tile.end;
    if (SPLIT || done == to) {
      done = 0;
      t += gridDim.x / CTAS;
    }
    return true;
  }
};

// 16 scale bytes from p on, of a row with `valid` bytes left, in a matrix that
// ends at `end`: as they lie, in the one or two 16-byte blocks around them (rows
// of scales start at any byte).  What follows the row's bytes is read by no
// instruction.  Blocks that the matrix's end cuts are read by bytes.
__device__ __forceinline__ void load_scales(uint4& lo, uint4& hi, const uint8_t* p, int valid,
                                            const uint8_t* end) {
  const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15;
  const uint4* block = reinterpret_cast<const uint4*>(p - shift);
  const bool two = shift + min(valid, 16) > 16;
  const bool cut = reinterpret_cast<const uint8_t*>(block + (two ? 2 : 1)) > end;
  lo = hi = make_uint4(0, 0, 0, 0);
  if (valid > 0 && !cut) {
    lo = __ldg(block);
    if (two) hi = __ldg(block + 1);
  }
  if (valid > 0 && cut) {
    uint32_t w[8] = {};
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= shift && i < shift + min(valid, 16))
        w[i / 4] |= static_cast<uint32_t>(__ldg(p - shift + i)) << (8 * (i % 4));
    lo = make_uint4(w[0], w[1], w[2], w[3]);
    hi = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// The 16 bytes from byte `shift` of two blocks on.
__device__ __forceinline__ uint4 shift_scales(uint4 lo, uint4 hi, uint32_t shift) {
  uint32_t w[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z};
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 2];
    w[5] = hi.w;
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const uint32_t bits = 8 * (shift & 3);
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Writes a warp's patch of 32 rows x 128 bytes (64 bf16 or 32 fp32 columns),
// staged in shared memory with 16-byte units swizzled by row, to `rows` rows of
// the output at `col`; `cols` columns exist.  Whole patches of 16-byte aligned
// rows leave as full 128-byte lines (four rows an instruction), others by
// elements, a row at a time.
template <bool F32>
__device__ __forceinline__ void store_patch(const GroupedArgs& a, uint32_t patch, int lane,
                                            int64_t row, int rows, int col, int cols, bool add) {
  constexpr int width = F32 ? 32 : 64;
  if (a.out_vec && cols >= width) {
    const int u = lane % 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + lane / 8;
      uint4 v = lds128(patch + r * 128 + ((u ^ (r & 7)) << 4));
      if (r < rows) {
        if constexpr (F32) {
          float* p = static_cast<float*>(a.out) + (row + r) * a.ldo + col + 4 * u;
          if (add) {
            const float4 o = *reinterpret_cast<const float4*>(p);
            v = make_uint4(__float_as_uint(__uint_as_float(v.x) + o.x),
                           __float_as_uint(__uint_as_float(v.y) + o.y),
                           __float_as_uint(__uint_as_float(v.z) + o.z),
                           __float_as_uint(__uint_as_float(v.w) + o.w));
          }
          stg128(p, v.x, v.y, v.z, v.w);
        } else {
          stg128(static_cast<uint16_t*>(a.out) + (row + r) * a.ldo + col + 8 * u, v.x, v.y, v.z,
                 v.w);
        }
      }
    }
    return;
  }
  // Eight rows are read before any is written, so that a row's way through shared
  // memory is not waited for 32 times (1013 rows over 5 experts, 1001 x 1056, fp32:
  // 13.0 us one by one, 9.8 so).
  constexpr int BATCH = 8;
  if constexpr (F32) {
    float* p = static_cast<float*>(a.out) + row * a.ldo + col + lane;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += BATCH) {
      float v[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        v[i] = __uint_as_float(
            lds32(patch + (r0 + i) * 128 + (((lane / 4) ^ (i & 7)) << 4) + lane % 4 * 4));
      if (add) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          if (r0 + i < rows && lane < cols) v[i] += p[i * a.ldo];
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (r0 + i < rows && lane < cols) p[i * a.ldo] = v[i];
      p += BATCH * a.ldo;
    }
    return;
  }
  // bf16: a lane a pair of columns that starts on 4 bytes, and the first or last
  // column by itself where the row's ends leave it over.
  uint16_t* p = static_cast<uint16_t*>(a.out) + row * a.ldo + col;
  const int limit = min(cols, 64), skew = static_cast<int>(a.ldo & 1);
  const int odd0 = static_cast<int>((reinterpret_cast<uintptr_t>(p) / 2) & 1);
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += BATCH) {
    uint32_t pair[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      pair[i] = lds32(patch + (r0 + i) * 128 + (((lane / 4) ^ (i & 7)) << 4) + lane % 4 * 4);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int odd = odd0 ^ (skew & i);
      const uint32_t v = pair[i], next = __shfl_down_sync(~0u, v, 1);
      const int c = 2 * lane + odd;
      if (r0 + i < rows) {
        if (c + 1 < limit) stg32(p + c, odd ? v >> 16 | next << 16 : v);
        if (odd && lane == 0 && limit > 0) p[0] = static_cast<uint16_t>(v);
        if (((limit - odd) & 1) && limit > odd && lane == (limit - 1) / 2)
          p[limit - 1] = static_cast<uint16_t>(limit & 1 ? v : v >> 16);
      }
      p += a.ldo;
    }
  }
}

// Floats of a row of a part of a FORWARD tile's sums in shared memory: lanes that
// write 16 bytes of neighbouring rows meet no bank twice.
constexpr int PART_LD = 128 + 4;

template <int CTAS, int BN, int KIND, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
mx_grouped_kernel(const __grid_constant__ GroupedMaps maps, const GroupedArgs a) {
  using S = Shape<CTAS, BN>;
  constexpr int CHUNK = S::CHUNK;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_up_shared<1024>(smem_raw);
  const uint32_t stages = smem_addr(smem);
  const uint32_t scales = stages + S::STAGES * S::STAGE_BYTES;
  const uint32_t patches = scales + S::SCALE_CHUNKS * S::SCALE_BYTES;
  int* off = reinterpret_cast<int*>(smem + S::STAGES * S::STAGE_BYTES +
                                    S::SCALE_CHUNKS * S::SCALE_BYTES + S::OUT_BYTES);
  int* start = off + GROUPS_MAX + 1;
  const uint32_t bars = smem_addr(start + GROUPS_MAX + 1);   // 8-byte aligned: 2 (MAX + 1) words
  const uint32_t full = bars, empty = full + 8 * S::STAGES;
  const uint32_t sc_full = empty + 8 * S::STAGES, sc_empty = sc_full + 8 * S::SCALE_CHUNKS;
  const uint32_t acc_full = sc_empty + 8 * S::SCALE_CHUNKS, acc_empty = acc_full + 16;
  const uint32_t drain = acc_empty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(start + GROUPS_MAX + 1) + 2 * S::BARRIERS;

  const int tid = threadIdx.x, lane = tid % 32;
  const int warp = __shfl_sync(~0u, tid / 32, 0);          // the same for the warp, known to be
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;   // 0: the CTA that issues

  // full, sc_full and acc_empty are waited on by the issuing CTA alone, and
  // with pairs the other CTA's copies and warps arrive there; the others are
  // each CTA's own.
  if (tid == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < S::SCALE_CHUNKS; ++i) {
      mbar_init(sc_full + 8 * i, 4 * CTAS);
      mbar_init(sc_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 4 * CTAS);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc<CTAS>(smem_addr(tmem_slot), TMEM_COLS);

  // Offsets, checked, and the groups' first tiles (scanned by one warp, 32
  // groups a step).
  bool bad = false;
  for (int i = tid; i <= a.groups; i += THREADS) {
    const int v = a.offsets[i];
    const int before = i > 0 ? a.offsets[i - 1] : 0;
    bad |= v < before || v > a.limit || (KIND == WGRAD && v % 32 != 0);
    off[i] = v;
  }
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    int total = 0;
    for (int i = 0; i < a.groups; i += 32) {
      int n = 0;
      if (!bad && i + lane < a.groups) {
        const int rows_g = off[i + lane + 1] - off[i + lane];
        const int rows = KIND == FORWARD ? rows_g : a.a_rows, cols = KIND == FEW ? rows_g : a.b_rows;
        n = (rows + ROWS * CTAS - 1) / (ROWS * CTAS) * ((cols + BN - 1) / BN);
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
  if constexpr (CTAS == 2) cluster_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  const int tile0 = static_cast<int>(blockIdx.x) / (SPLIT ? a.split : CTAS);
  Walk<CTAS, BN, KIND, SPLIT> walk{off, start, a.groups, tile0, 0, 0};
  Tile tile;
  bool ok = true;

  if (warp == 8) {
    // ---- copies: a stage of this CTA's rows of A and of B at a time ----
    if (elect_one()) {
      uint32_t it = 0;
      while (ok && walk.next(a, tile)) {
        const int ay = tile.ay + tile.m0 + static_cast<int>(rank) * ROWS;
        const int by = tile.by + tile.n0 + static_cast<int>(rank) * S::B_ROWS;
        for (int k = tile.step0(); k < tile.step1(); ++k, ++it) {
          const uint32_t s = it % S::STAGES;
          if (it >= S::STAGES &&
              !mbar_wait_bounded(empty + 8 * s, (it / S::STAGES - 1) & 1, a.timeout_ns)) {
            ok = false;
            break;
          }
          const uint32_t dst = stages + s * S::STAGE_BYTES, bar = full + 8 * s;
          if (rank == 0) mbar_arrive_expect_tx(bar, CTAS * S::STAGE_BYTES);
          const int x = k * STEP_K;
          if constexpr (CTAS == 2) {
            const uint32_t there = cluster_addr(bar, 0);
            tma_load_3d_pair(dst, &maps.a, x, ay, tile.az, there);
            tma_load_3d_pair(dst + S::A_BYTES, &maps.b, x, by, tile.bz, there);
          } else {
            tma_load_3d(dst, &maps.a, x, ay, tile.az, bar);
            tma_load_3d(dst + S::A_BYTES, &maps.b, x, by, tile.bz, bar);
          }
        }
      }
      // After a wait that ran out, the copies in flight still land (a pair's
      // second CTA stays until its first has seen that).
      if (!ok && rank == 0)
        for (uint32_t i = it > S::STAGES ? it - S::STAGES : 0; i < it; ++i)
          mbar_wait_bounded(full + 8 * (i % S::STAGES), (i / S::STAGES) & 1, a.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---- tensor-core instructions, from one thread ----
    if (rank == 0 && elect_one()) {
      uint32_t it = 0, chunk = 0, acc = 0;
      while (ok && walk.next(a, tile)) {
        const int k0 = tile.step0(), k1 = tile.step1();
        if (k0 == k1) continue;
        // The accumulator's columns are free: for 256 columns, the shared 32
        // of the tile before (whose readers have then finished the tile
        // before that); otherwise, all of the tile two before.
        const uint32_t lag = BN == 256 ? 1 : 2;
        if (acc >= lag && !mbar_wait_bounded_cluster(acc_empty + 8 * ((acc - lag) % 2),
                                                     ((acc - lag) / 2) & 1, a.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem + S::acc_col(acc % 2);
        bool accumulate = false;
        for (int k = k0; ok && k < k1; ++k, ++it) {
          const uint32_t c = chunk % S::SCALE_CHUNKS, s = it % S::STAGES;
          if ((k == k0 || k % CHUNK == 0) &&
              !mbar_wait_bounded_cluster(sc_full + 8 * c, (chunk / S::SCALE_CHUNKS) & 1,
                                         a.timeout_ns))
            ok = false;
          if (!ok || !mbar_wait_bounded(full + 8 * s, (it / S::STAGES) & 1, a.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          // Scales of this stage: A's tile, then B's, in alternating columns.
          const uint32_t sc = scales + c * S::SCALE_BYTES + (k % CHUNK) * 512;
          const uint32_t ts = tmem + SCALE_COL + (k % 2) * 16;
          tc_copy_scales<CTAS>(ts, scale_desc(sc));
#pragma unroll
          for (int b = 0; b < S::B_TILES; ++b)
            tc_copy_scales<CTAS>(ts + 4 + 4 * b, scale_desc(sc + (1 + b) * CHUNK * 512));
          const uint64_t da = operand_desc(stages + s * S::STAGE_BYTES);
          const uint64_t db = operand_desc(stages + s * S::STAGE_BYTES + S::A_BYTES);
          const int j0 = (tile.first - k * STEP_K) / 32, j1 = (tile.end - k * STEP_K) / 32;
#pragma unroll
          for (int j = 0; j < STEP_K / 32; ++j)
            if (j >= j0 && j < j1) {
              tc_mma_mxf8<CTAS>(d, da + 2 * j, db + 2 * j, mxf8_idesc(ROWS * CTAS, BN, j), ts,
                                ts + 4, accumulate);
              accumulate = true;
            }
          tc_commit<CTAS>(empty + 8 * s);
          if (k % CHUNK == CHUNK - 1 || k == k1 - 1) {
            tc_commit<CTAS>(sc_empty + 8 * c);
            ++chunk;
          }
        }
        if (ok) tc_commit<CTAS>(acc_full + 8 * (acc % 2));
        ++acc;
      }
      // Nothing of this thread's is in flight when the memory is given back.
      if (!ok) {
        tc_commit<CTAS>(drain);
        mbar_wait_bounded(drain, 0, a.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---- scales: thread t takes piece t % 4 of rows t / 4 + 32 i of this
    // CTA's A rows and of all of B's, so that a row's 64 bytes are one request,
    // and a thread's rows one 16-byte unit of each stage's tile.  A window's loads
    // are all in flight at once, and then its stores wait for places; a second
    // window does not fit the registers. ----
    const int piece = tid % 4, r = (tid - 128) / 4;
    const int64_t a_total = KIND == FORWARD ? a.limit
                            : KIND == FEW   ? static_cast<int64_t>(a.groups) * a.a_rows : a.a_rows;
    const int64_t b_total = KIND == FORWARD ? static_cast<int64_t>(a.groups) * a.b_rows
                            : KIND == FEW   ? a.limit : a.b_rows;
    const uint8_t* a_end = a.a_s + a_total * a.s_ld;
    const uint8_t* b_end = a.b_s + b_total * a.s_ld;
    const bool whole = a.s_ld % 16 == 0;     // every piece is a 16-byte block
    const uint8_t *ap = nullptr, *bp = nullptr;
    int at = 0, end = 0;             // scale bytes of the tile being loaded
    int a_left = 0, b_left = 0;      // rows from r on that exist
    auto row_scales = [&](int b, int i) {
      return b == 0 ? ap + i * 32 * a.s_ld : bp + ((b - 1) * 128 + i * 32) * a.s_ld;
    };
    // A window's scales, the blocks after them where pieces are not whole ones, its
    // first stage, its tile's, and where the first rows start in 16-byte blocks.
    struct Window {
      uint4 v[1 + S::B_TILES][4], hi[1 + S::B_TILES][4];
      int step, first, end;
      uint32_t a_shift, b_shift;
    };
    uint32_t chunk = 0;
    // Apart where pieces are whole blocks, so that the others' second blocks and
    // shifts are not in this loop's way (wgrad 16384 x 14336 x 4096 over 8 experts 712
    // -> 684 us, 6656 x 1024 x 6272 over 37 206 -> 177).
    auto run = [&](auto aligned) {
      constexpr bool WHOLE = decltype(aligned)::value;
      auto load = [&](Window& w) {
        while (at >= end) {
          if (!walk.next(a, tile)) return false;
          const int row = tile.m0 + static_cast<int>(rank) * ROWS + r;
          at = tile.step0() / WINDOW * (WINDOW * 4);
          end = tile.first < tile.end ? tile.end / 32 : at;
          a_left = tile.rows - row;
          b_left = min(tile.cols - tile.n0, BN) - r;
          ap = a.a_s + (static_cast<int64_t>(tile.az) * a.a_rows + tile.ay + row) * a.s_ld + 16 * piece;
          bp = a.b_s + (static_cast<int64_t>(tile.bz) * a.b_rows + tile.by + tile.n0 + r) * a.s_ld +
               16 * piece;
        }
        // Pieces before the range are skipped like those after it.
        const int valid = at + 16 * piece + 16 > tile.first / 32 ? end - at - 16 * piece : 0;
        // All loads are asked for before any is waited for.
#pragma unroll
        for (int b = 0; b <= S::B_TILES; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint8_t* p = row_scales(b, i) + at;
            const int has = (b == 0 ? 32 * i < a_left : (b - 1) * 128 + 32 * i < b_left) ? valid : 0;
            if constexpr (WHOLE)
              w.v[b][i] = has > 0 ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
            else
              load_scales(w.v[b][i], w.hi[b][i], p, has, b == 0 ? a_end : b_end);
          }
        w.step = at / 4;
        w.first = tile.step0();
        w.end = tile.step1();
        w.a_shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(ap)) & 15;
        w.b_shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(bp)) & 15;
        at += WINDOW * 4;
        return true;
      };
      auto store = [&](Window& w) {
#pragma unroll
        for (int h = 0; h < WINDOW / CHUNK; ++h) {
          if (w.step + (h + 1) * CHUNK <= w.first || w.step + h * CHUNK >= w.end) continue;
          const uint32_t c = chunk % S::SCALE_CHUNKS;
          if (chunk >= S::SCALE_CHUNKS &&
              !mbar_wait_bounded(sc_empty + 8 * c, (chunk / S::SCALE_CHUNKS - 1) & 1, a.timeout_ns)) {
            ok = false;
            break;
          }
          ++chunk;
          constexpr int PIECES = CHUNK / 4;
          if (piece / PIECES == h) {
            const uint32_t dst = scales + c * S::SCALE_BYTES + piece % PIECES * 2048 + r * 16;
#pragma unroll
            for (int b = 0; b <= S::B_TILES; ++b) {
              if constexpr (!WHOLE) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint32_t rows = b == 0 ? 32 * i : (b - 1) * 128 + 32 * i;
                  w.v[b][i] = shift_scales(
                      w.v[b][i], w.hi[b][i],
                      ((b == 0 ? w.a_shift : w.b_shift) + rows * static_cast<uint32_t>(a.s_ld)) & 15);
                }
              }
              const uint32_t to = dst + b * CHUNK * 512;
              sts128(to, w.v[b][0].x, w.v[b][1].x, w.v[b][2].x, w.v[b][3].x);
              sts128(to + 512, w.v[b][0].y, w.v[b][1].y, w.v[b][2].y, w.v[b][3].y);
              sts128(to + 1024, w.v[b][0].z, w.v[b][1].z, w.v[b][2].z, w.v[b][3].z);
              sts128(to + 1536, w.v[b][0].w, w.v[b][1].w, w.v[b][2].w, w.v[b][3].w);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            if constexpr (CTAS == 2) mbar_arrive_cluster(cluster_addr(sc_full + 8 * c, 0));
            else mbar_arrive(sc_full + 8 * c);
          }
        }
      };
      Window w;
      while (ok && load(w)) store(w);
    };
    if (whole) run(std::true_type{});
    else run(std::false_type{});
  } else {
    // ---- epilogue: warp w reads lanes 32 w .. 32 w + 31, a row each ----
    uint32_t acc = 0, turn = 0;
    while (ok && walk.next(a, tile)) {
      const int first = tile.m0 + static_cast<int>(rank) * ROWS + warp * 32;
      const int rows = min(32, tile.rows - first);       // may be negative
      const int64_t out_row = first + (KIND == WGRAD ? static_cast<int64_t>(tile.g) * a.a_rows
                                                     : static_cast<int64_t>(tile.ay));
      const uint32_t s = acc % 2;
      const bool empty_tile = tile.first == tile.end;
      // Whole patches leave by bulk copies, clipped at the output's last column
      // (later ranges are added there: what a warp has written before is
      // complete); those with rows of the next group, by threads.
      const bool bulk = KIND != FEW && a.out_vec && (KIND == WGRAD ? rows > 0 : rows == 32);
      if (tile.add && lane == 0) bulk_wait_all();
      if (!empty_tile) {
        if (!mbar_wait_bounded(acc_full + 8 * s, (acc / 2) & 1, a.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        ++acc;
      }
      if constexpr (SPLIT) {
        // The range's sums, where the stages were: columns of 128 rows (FEW), rows of
        // PART_LD columns.  The tile's instructions, its last, are complete.
        const uint32_t from = tmem + S::acc_col(s) + (static_cast<uint32_t>(warp) << 21);
        const int r = warp * 32 + lane;
#pragma unroll 1
        for (int j = 0; j < BN; j += 32) {
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = 0;
          if (!empty_tile) {
            tmem_load_x32(from + j, v);
            tmem_wait_load();
          }
          if constexpr (KIND == FEW) {
#pragma unroll
            for (int c = 0; c < 32; ++c) sts32(stages + ((j + c) * ROWS + r) * 4, v[c]);
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 4)
              sts128(stages + (r * PART_LD + j + c) * 4, v[c], v[c + 1], v[c + 2], v[c + 3]);
          }
        }
        continue;
      } else if constexpr (KIND == FEW) {
        // The lanes hold 32 neighbouring columns of a row of the output, row by row.
        const uint32_t from = tmem + S::acc_col(s) + (static_cast<uint32_t>(warp) << 21);
#pragma unroll 1
        for (int j = 0; j < BN; j += 32) {
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = 0;
          if (!empty_tile) {
            tmem_load_x32(from + j, v);
            tmem_wait_load();
          }
          tc_fence_before_sync();
          __syncwarp();
          if (!empty_tile && lane == 0 && j == BN - 32) mbar_arrive(acc_empty + 8 * s);
          const int count = lane < rows ? tile.cols - tile.n0 - j : 0;
          const int64_t at = (static_cast<int64_t>(tile.by) + tile.n0 + j) * a.ldo + first + lane;
          if (a.out_f32) {
            float* p = static_cast<float*>(a.out) + at;
            if (tile.add) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c < count) v[c] = __float_as_uint(__uint_as_float(v[c]) + p[c * a.ldo]);
            }
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c < count) p[c * a.ldo] = __uint_as_float(v[c]);
          } else {
            uint16_t* p = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c < count)
                p[c * a.ldo] = static_cast<uint16_t>(pack_bf16(__uint_as_float(v[c]), 0.f));
          }
        }
        continue;
      }
      const int width = a.out_f32 ? 32 : 64;             // columns of a patch
      if (empty_tile && bulk) {
        // One patch of zeros for all the columns.
        const uint32_t patch = patches + (warp * S::PATCHES + turn++ % (S::PATCHES ? S::PATCHES : 1)) * 4096;
        if (lane == 0) bulk_wait_read<S::PATCHES ? S::PATCHES - 1 : 0>();
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) sts128(patch + u * 512 + lane * 16, 0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          for (int j = 0; j < BN && tile.n0 + j < tile.cols; j += width)
            tma_store_3d(&maps.out, patch, tile.n0 + j, KIND == WGRAD ? first : static_cast<int>(out_row),
                         KIND == WGRAD ? tile.g : 0);
          bulk_commit();
        }
        continue;
      }
      const uint32_t base = tmem + S::acc_col(s) + (static_cast<uint32_t>(warp) << 21);
      // The loop for each way out and type, so that the one of whole patches, which
      // bounds short contractions, stays small.
      auto drain = [&](auto whole, auto wide) {
        constexpr bool BULK = decltype(whole)::value, F32 = decltype(wide)::value;
        constexpr int WIDTH = F32 ? 32 : 64;             // columns of a patch
#pragma unroll 1
        for (int i = 0; i < BN; i += WIDTH) {
          // Accumulator 0 shares its last 32 columns with the next tile's
          // first 32: they are read first.
          const int j = BN == 256 && s == 0 ? BN - WIDTH - i : i;
          const uint32_t patch =
              patches + (warp * S::PATCHES + turn++ % (S::PATCHES ? S::PATCHES : 1)) * 4096;
          if (lane == 0) bulk_wait_read<S::PATCHES ? S::PATCHES - 1 : 0>();
          __syncwarp();
#pragma unroll
          for (int h = 0; h < WIDTH / 32; ++h) {
            uint32_t v[32];
            if (!BULK && empty_tile) {
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = 0;
            } else {
              tmem_load_x32(base + j + 32 * h, v);
              tmem_wait_load();
              // The columns that the next tile waits for have been read.
              if (i == (BN == 256 ? 0 : BN - WIDTH) && h == WIDTH / 32 - 1) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                  if constexpr (CTAS == 2) mbar_arrive_cluster(cluster_addr(acc_empty + 8 * s, 0));
                  else mbar_arrive(acc_empty + 8 * s);
                }
              }
            }
            const uint32_t line = patch + lane * 128;
            if constexpr (F32) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                sts128(line + ((u ^ (lane & 7)) << 4), v[4 * u], v[4 * u + 1], v[4 * u + 2],
                       v[4 * u + 3]);
            } else {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                uint32_t w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  w[c] = pack_bf16(__uint_as_float(v[8 * u + 2 * c]),
                                   __uint_as_float(v[8 * u + 2 * c + 1]));
                sts128(line + (((4 * h + u) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if constexpr (!BULK) {
            store_patch<F32>(a, patch, lane, out_row, rows, tile.n0 + j, tile.cols - tile.n0 - j,
                             tile.add);
          } else if (lane == 0 && tile.n0 + j < tile.cols) {
            const int y = KIND == WGRAD ? first : static_cast<int>(out_row);
            const int z = KIND == WGRAD ? tile.g : 0;
            if (F32 && tile.add) tma_add_3d(&maps.out, patch, tile.n0 + j, y, z);
            else tma_store_3d(&maps.out, patch, tile.n0 + j, y, z);
          }
          if (lane == 0) bulk_commit();       // one group a patch, empty ones too
        }
      };
      if (bulk && a.out_f32) drain(std::true_type{}, std::true_type{});
      else if (bulk) drain(std::true_type{}, std::false_type{});
      else if (a.out_f32) drain(std::false_type{}, std::true_type{});
      else drain(std::false_type{}, std::false_type{});
    }
    if (lane == 0) bulk_wait_all();
  }

  if (!ok && a.dev_err) atomicOr(a.dev_err, MXQ_DEVERR_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (SPLIT) {
    // Every CTA adds its share of the tile, the ranges in order.
    cluster_sync();
    Walk<CTAS, BN, KIND, SPLIT> again{off, start, a.groups, tile0, 0, 0};
    if (again.next(a, tile)) {
      const int part = static_cast<int>(cluster_rank());
      const int rows = min(ROWS, tile.rows - tile.m0), cols = min(BN, tile.cols - tile.n0);
      if constexpr (KIND == FEW) {
        const int r = tid % ROWS;
        constexpr int AT_ONCE = THREADS / ROWS;
        if (tid < AT_ONCE * ROWS && r < rows) {
#pragma unroll 2
          for (int c = tid / ROWS * a.split + part; c < cols; c += AT_ONCE * a.split) {
            const uint32_t at = stages + (c * ROWS + r) * 4;
            float v[SPLIT_MAX], sum = 0;
#pragma unroll
            for (int p = 0; p < SPLIT_MAX; ++p) v[p] = p < a.split ? ld_cluster_f32(at, p) : 0.f;
#pragma unroll
            for (int p = 0; p < SPLIT_MAX; ++p) sum += v[p];
            const int64_t to = (static_cast<int64_t>(tile.by) + tile.n0 + c) * a.ldo + tile.m0 + r;
            if (a.out_f32) static_cast<float*>(a.out)[to] = sum;
            else
              static_cast<uint16_t*>(a.out)[to] = static_cast<uint16_t>(pack_bf16(sum, 0.f));
          }
        }
      } else {
#pragma unroll 1
        for (int r = warp * a.split + part; r < rows; r += THREADS / 32 * a.split) {
          const uint32_t at = stages + (r * PART_LD + 4 * lane) * 4;
          float4 v[SPLIT_MAX];
#pragma unroll
          for (int p = 0; p < SPLIT_MAX; ++p)
            v[p] = p < a.split ? ld_cluster_f32x4(at, p) : make_float4(0.f, 0.f, 0.f, 0.f);
          float sum[4] = {};
#pragma unroll
          for (int p = 0; p < SPLIT_MAX; ++p) {
            sum[0] += v[p].x;
            sum[1] += v[p].y;
            sum[2] += v[p].z;
            sum[3] += v[p].w;
          }
          const int left = cols - 4 * lane;
          const int64_t row = KIND == WGRAD ? static_cast<int64_t>(tile.g) * a.a_rows
                                            : static_cast<int64_t>(tile.ay);
          const int64_t to = (row + tile.m0 + r) * a.ldo + tile.n0 + 4 * lane;
          if (a.out_f32) {
            float* p = static_cast<float*>(a.out) + to;
            if (a.out_vec && left >= 4) {
              *reinterpret_cast<float4*>(p) = make_float4(sum[0], sum[1], sum[2], sum[3]);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (c < left) p[c] = sum[c];
            }
          } else {
            uint16_t* p = static_cast<uint16_t*>(a.out) + to;
            const uint32_t lo = pack_bf16(sum[0], sum[1]), hi = pack_bf16(sum[2], sum[3]);
            if (a.out_vec && left >= 4) {
              *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (c < left) p[c] = static_cast<uint16_t>((c < 2 ? lo : hi) >> (c % 2 * 16));
            }
          }
        }
      }
    }
  }
  // A cluster's CTAs leave together: each arrives on the other's barriers, or reads
  // its sums.
  if constexpr (CTAS == 2 || SPLIT) cluster_sync();
  tc_fence_after_sync();
  if (warp == 9) tmem_dealloc<CTAS>(tmem, TMEM_COLS);
}

// CTAs that share a tile's contraction, of `depth` values on average and `most` at
// most, where there are fewer tiles than SMs (of which clusters of four reach 144).
int ranges(int64_t depth, int64_t most, int64_t tiles, bool out_f32, int num_sms) {
  const int64_t steps = (depth + STEP_K - 1) / STEP_K;
  int split = 1;
  while (split < SPLIT_MAX && steps >= 4 * SPLIT_STEPS && steps >= 2 * split * SPLIT_STEPS &&
         tiles * 2 * split * 64 <= num_sms * (64 - 2 * split))
    split *= 2;
  // Sums of more than SEGMENT values are taken apart by the other kernel.
  const int64_t each = ((most + STEP_K - 1) / STEP_K + split) / split * STEP_K;
  return out_f32 && each > SEGMENT + STEP_K ? 1 : split;
}

template <int CTAS, int BN, int KIND, bool SPLIT = false>
cudaError_t launch(const GroupedMaps& maps, const GroupedArgs& a, const GroupedPlan& plan,
                   cudaStream_t stream) {
  auto kernel = mx_grouped_kernel<CTAS, BN, KIND, SPLIT>;
  constexpr int smem = Shape<CTAS, BN>::SMEM;
  static_assert(smem <= 227 * 1024, "shared memory of one SM");
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), smem, &allowed);
  if (e != cudaSuccess) return e;
  const int cluster = SPLIT ? plan.split : CTAS;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.grid));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

template <int KIND>
cudaError_t launch_plan(const GroupedMaps& maps, const GroupedArgs& a, const GroupedPlan& plan,
                        cudaStream_t stream) {
  if (plan.ctas == 2) return launch<2, 256, KIND>(maps, a, plan, stream);
  if (plan.cols == 256) return launch<1, 256, KIND>(maps, a, plan, stream);
  return plan.split > 1 ? launch<1, 128, KIND, true>(maps, a, plan, stream)
                        : launch<1, 128, KIND>(maps, a, plan, stream);
}

// The cut with the least estimated time: waves of tiles over the GPU, each so
// many clocks a stage and so many more, as measured with all SMs at work (128
// columns 460 and 2500, 256 columns 720 and 5000, pairs of CTAs 620 and 7000).
// Pairs read the fewest bytes of codes a product and win large calls (gemm 16384
// x 14336 x 4096 over 8 experts 657 us, 682 in 256 columns, 856 in 128), the
// others where its tiles fill the GPU worse (4096 x 2048 x 2048 over 8 experts
// 25.6, 21.8 and 25.5 us).  A contraction of four stages or less leaves the
// epilogue alone to bound the call, and two whole accumulators of 128 columns
// keep it busiest (weight gradients of 64 experts x 1408 x 2048 from 128 rows
// each 200, 166 and 147 us).  For groups of rows / groups output rows on average.
GroupedPlan cut(int64_t rows, int64_t cols, int64_t depth, int64_t groups, bool wgrad,
                int num_sms) {
  if (!wgrad && rows <= groups * FEW_ROWS) return {1, 32, true};
  if (depth <= 4 * STEP_K) return {1, 128, false};
  auto clocks = [&](int ctas, int bn, int stage, int fixed) {
    const int64_t tile = ROWS * ctas;
    const int64_t tiles_m = wgrad ? groups * ((rows / groups + tile - 1) / tile)
                                  : rows / tile + (groups + 1) / 2;
    const int64_t tiles = tiles_m * ((cols + bn - 1) / bn), at_once = num_sms / ctas;
    return (tiles + at_once - 1) / at_once * ((depth + STEP_K - 1) / STEP_K * stage + fixed);
  };
  const int64_t narrow = clocks(1, 128, 460, 2500), wide = clocks(1, 256, 720, 5000),
                pair = clocks(2, 256, 620, 7000);
  if (narrow <= wide && narrow <= pair) return {1, 128, false};
  return {pair <= wide ? 2 : 1, 256, false};
}

}  // namespace

GroupedPlan grouped_plan(int64_t M, int64_t N, int64_t K, int64_t groups, bool wgrad,
                         bool out_f32, int num_sms) {
  GroupedPlan plan = wgrad ? cut(N * groups, K, M / groups, groups, true, num_sms)
                           : cut(M, N, K, groups, false, num_sms);
  // At most this many tiles, whatever the offsets are: every group has a row more
  // than whole tiles.
  const int64_t used = groups < M ? groups : M;
  auto ragged = [&](int tile) { return (M - used) / tile + used; };
  auto whole = [](int64_t n, int tile) { return (n + tile - 1) / tile; };
  const int tile_m = ROWS * plan.ctas;
  plan.tiles = wgrad      ? groups * whole(N, tile_m) * whole(K, plan.cols)
               : plan.few ? ragged(plan.cols) * whole(N, tile_m)
                          : ragged(tile_m) * whole(N, plan.cols);
  plan.split = plan.cols == 256 ? 1
               : wgrad          ? ranges(M / groups, M, plan.tiles, out_f32, num_sms)
                                : ranges(K, K, plan.tiles, out_f32, num_sms);
  const int cluster = plan.split > 1 ? plan.split : plan.ctas;
  const int64_t most = num_sms / cluster;
  plan.grid = static_cast<int>(plan.tiles < most ? plan.tiles : most) * cluster;
  return plan;
}

cudaError_t launch_grouped(const GroupedMaps& maps, const GroupedArgs& a, bool wgrad,
                           const GroupedPlan& plan, cudaStream_t stream) {
  if (plan.few)
    return plan.split > 1 ? launch<1, 32, FEW, true>(maps, a, plan, stream)
                          : launch<1, 32, FEW>(maps, a, plan, stream);
  return wgrad ? launch_plan<WGRAD>(maps, a, plan, stream)
               : launch_plan<FORWARD>(maps, a, plan, stream);
}

}  // namespace mxq
