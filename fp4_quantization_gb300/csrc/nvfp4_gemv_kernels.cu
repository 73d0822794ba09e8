// nvfp4_gemv_kernels.cu -- few rows times NVFP4 weights.
//
// out[r, n] = G_e * sum_k x[r / share, k] * s[n, k / 16] * c[n, k] for the
// expert e of row r, with E2M1 codes c, E4M3 scales s and the fp32 scale G_e.
//
// Bound by reading the weights once (9/16 byte a weight).  The products run
// on the warp-level tensor instruction (m16n8k16, f16 in, fp32 sums): with
// few rows the weights are its 16-row operand straight from registers, so a
// weight costs half a conversion, half a multiply by its block scale and
// 1/128 of an instruction for up to 8 rows of x, where fp32 multiply-adds
// would cost three more instructions a weight.  Both operands are exact:
//  * s * c has at most 6 significant bits and lies in 2^-10 .. 2688: an f16.
//  * x is taken in windows of 29 binades from each row's largest magnitude
//    down; scaled by a power of two that puts the largest in 2^14 .. 2^15, a
//    window's bf16 values are normal f16 numbers.  One window holds a row
//    unless its magnitudes spread over more than 2^28; otherwise the weights
//    are read again for the next window.
#include "mxq_products.h"

#include "mxq_tc_ptx.cuh"

namespace mxq {
namespace {

constexpr int WARPS = 8;
constexpr int STEP_K = 256;          // K of one step of a warp: a line of codes a row
constexpr int STEP_BYTES = 16 * STEP_K / 2;
constexpr int SUM_BYTES = 8 * 1024;  // partial sums of some items
constexpr int BATCH = 4;             // 16-byte loads of x in flight a thread

// Rows of x at a time: up to 8 or 16.  Two CTAs share an SM.
template <int TOKS>
struct Shape {
  static constexpr int TILES = TOKS / 8;                 // of 8 columns of the instruction
  static constexpr int DEPTH = TOKS == 16 ? 3 : 4;       // steps of a warp in shared memory
  static constexpr int RING_BYTES = WARPS * DEPTH * STEP_BYTES;
  static constexpr int X_BYTES = (TOKS == 16 ? 44 : 28) * 1024;   // staged rows of x
  static constexpr int SMEM = RING_BYTES + X_BYTES + SUM_BYTES + 1024;
};

__device__ __forceinline__ void store_out(const GemvArgs& a, int64_t row, int n, float v) {
  if (a.out_f32) {
    static_cast<float*>(a.out)[row * a.ldo + n] = v;
  } else {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(0.f), "f"(v));
    static_cast<uint16_t*>(a.out)[row * a.ldo + n] = static_cast<uint16_t>(d);
  }
}

// 8 E2M1 codes -> 4 pairs of f16, element 2i in the low half of pair i.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
  return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, __half2 b) {
  const __half2 d = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&d);
}

// A pair of bf16 values, each 0 unless its magnitude's bits are in [low, lim).
__device__ __forceinline__ uint32_t in_window(uint32_t pair, uint32_t low, uint32_t lim) {
  const uint32_t lo = pair & 0x7FFF, hi = (pair >> 16) & 0x7FFF;
  return (lo >= low && lo < lim ? pair & 0xFFFF : 0) |
         (hi >= low && hi < lim ? pair & 0xFFFF0000 : 0);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// A step's codes come by one tensor copy (16 rows of 128 bytes, 16-byte units
// swizzled by row), so that what is in flight costs neither registers nor the
// warps' load path; its scales are 4 bytes a thread and row.
//
// One step: codes at `ws`, the block scales of k = 64 t .. 64 t + 63 of rows g
// and g + 8 in s, and row g (and g + 8) of x at those k in 8 pieces of 16 bytes,
// x_step apart (0, at zeros, where there is no such row).  Thread (g, t)
// multiplies weight rows g and g + 8 by them; the instruction's k order is the
// codes' order, on both sides.
template <int TOKS>
__device__ __forceinline__ void multiply_step(float (&acc)[2][Shape<TOKS>::TILES][4], uint32_t ws,
                                              const uint32_t (&s)[2],
                                              const uint32_t (&x_at)[Shape<TOKS>::TILES],
                                              const uint32_t (&x_step)[Shape<TOKS>::TILES], int g,
                                              int t) {
  uint4 c[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      c[h][i] = lds128(ws + (g + 8 * h) * 128 + (((2 * t + i) ^ g) << 4));
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    __half2 sc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t pair = e4m3x2_to_f16(b < 2 ? s[h] & 0xFFFF : s[h] >> 16);
      const __half2 two = *reinterpret_cast<const __half2*>(&pair);
      sc[h] = b % 2 ? __high2half2(two) : __low2half2(two);
    }
#pragma unroll
    for (int p = 2 * b; p < 2 * b + 2; ++p) {
      uint4 x[Shape<TOKS>::TILES];
#pragma unroll
      for (int m = 0; m < Shape<TOKS>::TILES; ++m) {
        x[m] = lds128(x_at[m] + p * x_step[m]);
      }
      uint32_t v[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        e2m1x8_to_f16(word(c[h][p / 4], p % 4), v[h]);
#pragma unroll
        for (int n = 0; n < 4; ++n) v[h][n] = mul_f16x2(v[h][n], sc[h]);
      }
#pragma unroll
      for (int m = 0; m < Shape<TOKS>::TILES; ++m) {
        mma_f16(acc[0][m], v[0][0], v[1][0], v[0][1], v[1][1], x[m].x, x[m].y);
        mma_f16(acc[1][m], v[0][2], v[1][2], v[0][3], v[1][3], x[m].z, x[m].w);
      }
    }
  }
}

// Persistent CTAs (clusters of them) take an equal share each of the items
// (an expert that has rows, 16 * tiles of its output columns) in order, so
// that a CTA stages its rows of x once for many items.  A CTA's 8 warps are
// `tiles` tiles of 16 columns x 8 / tiles parts of K (taken step by step in
// turn); a cluster's CTAs split K into ranges.  The parts leave their sums in
// shared memory; when its places are full, or the rows of x change, they are
// added in a fixed order, and those of a cluster's CTAs by its first one.
//
// K is staged in chunks of what fits of the rows: of `cap`, or with UNEVEN of those
// that the pass has, so that an expert with few rows keeps them staged while another
// with many takes them in one pass over its weights.
template <int TOKS, bool UNEVEN>
__global__ void __launch_bounds__(32 * WARPS, 2)
nvfp4_gemv_kernel(const __grid_constant__ CUtensorMap codes, const GemvArgs a, const int tiles,
                  const int cluster, const int cap) {
  using S = Shape<TOKS>;
  constexpr int DEPTH = S::DEPTH, TILES = S::TILES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_up_shared<1024>(smem_raw);
  float* red = reinterpret_cast<float*>(smem + S::RING_BYTES);   // [item][warp][row][16]
  const uint32_t xs = smem_addr(smem + S::RING_BYTES + SUM_BYTES);
  __shared__ uint32_t present[GEMV_EXPERTS_MAX / 32];
  __shared__ uint16_t active[GEMV_EXPERTS_MAX];           // the experts that have rows
  __shared__ int warp_sum[WARPS];
  // Rows of the expert, their number, the next; whether its first room is another.
  __shared__ int list[TOKS + 3];
  __shared__ uint32_t extent[TILES * WARPS];               // of a warp's share of a row of x
  __shared__ uint64_t full[WARPS][DEPTH], empty[WARPS][DEPTH];   // of a part's places
  __shared__ uint4 zeros[1];
  __shared__ int rooms[2];                                // UNEVEN: of this pass, of its expert's first
  __shared__ float2 unit[TOKS];                           // what a sum of staged row i is multiplied by
  const int tid = threadIdx.x, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int warp = __shfl_sync(~0u, tid / 32, 0);          // the same for the warp, known to be
  const int rank = blockIdx.x % cluster;
  const int groups = (a.n + tiles * 16 - 1) / (tiles * 16);

  // Which experts have rows; rows without an expert are zero.
  int experts = 1;
  if (a.experts) {
    const int words = (a.num_experts + 31) / 32;
    static_assert(GEMV_EXPERTS_MAX / 32 <= 32 * WARPS, "a word a thread");
    if (tid < words) present[tid] = 0;
    __syncthreads();
#pragma unroll 1
    for (int r0 = warp * 32; r0 < a.rows; r0 += 32 * WARPS) {
      const int id = r0 + lane < a.rows ? a.experts[r0 + lane] : 0;
      const bool none = id < 0 || id >= a.num_experts;
      if (r0 + lane < a.rows && !none) atomicOr(&present[id / 32], 1u << (id % 32));
      for (uint32_t m = __ballot_sync(~0u, none); m; m &= m - 1)
        for (int n = blockIdx.x * 32 + lane; n < a.n; n += gridDim.x * 32)
          store_out(a, r0 + __ffs(m) - 1, n, 0.f);
    }
    __syncthreads();
    const uint32_t mine = tid < words ? present[tid] : 0;
    int sum = __popc(mine);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int up = __shfl_up_sync(~0u, sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int at = sum - __popc(mine);
    experts = 0;
#pragma unroll 1
    for (int i = 0; i < (words + 31) / 32; ++i) {
      if (i < warp) at += warp_sum[i];
      experts += warp_sum[i];
    }
    for (uint32_t m = mine; m; m &= m - 1)
      active[at++] = static_cast<uint16_t>(tid * 32 + __ffs(m) - 1);
    __syncthreads();
  }
  const int items = experts * groups;
  const int clusters = gridDim.x / cluster, me = blockIdx.x / cluster;
  const int each = items / clusters, extra = items % clusters;
  const int item_first = me * each + min(me, extra), item_end = item_first + each + (me < extra);
  if (item_first == item_end) return;

  // This CTA's range of K, and this warp's steps in it.
  const int parts = WARPS / tiles, tile = warp % tiles, part = warp / tiles;
  const int steps = (a.k + STEP_K - 1) / STEP_K, range = (steps + cluster - 1) / cluster;
  const int k_first = min(rank * range, steps) * STEP_K;
  const int k_end = min(min((rank + 1) * range, steps) * STEP_K, a.k);
  struct Item {
    int e, n0;            // its expert and first output column
  };
  auto item_at = [&](int i) {
    const int nth = a.experts ? i / groups : 0;
    return Item{a.experts ? static_cast<int>(active[nth]) : 0, (i - nth * groups) * tiles * 16};
  };
  // A warp's steps in the chunk from k0 on start at start_of(k0).
  auto room_for = [&](int rows) { return S::X_BYTES / (rows * 2) / STEP_K * STEP_K; };
  const int even = room_for(cap);
  auto room_of = [&](int i) { return UNEVEN ? rooms[i] : even; };
  const int turn = parts * STEP_K;
  auto start_of = [&](int k0) {
    const int behind = (k0 - k_first - part * STEP_K) % turn;
    return behind <= 0 ? k0 - behind : k0 + turn - behind;
  };
  // A part's loads: DEPTH steps (or places for them) at a time, in order over the
  // chunks and the items; its first warp asks for the codes of all its tiles in
  // one copy (a copy takes 110 clocks to issue, 2 KB at a time 18 bytes a clock),
  // each warp for its scales.
  const uint32_t ring = smem_addr(smem) + part * (DEPTH * tiles * STEP_BYTES);
  const uint32_t fulls = smem_addr(&full[part][0]), empties = smem_addr(&empty[part][0]);
  if (tid < parts) {
    for (int i = 0; i < DEPTH; ++i) {
      mbar_init(smem_addr(&full[tid][i]), 1);
      mbar_init(smem_addr(&empty[tid][i]), tiles);
    }
    fence_barrier_init();
  }
  if (tid == 0) zeros[0] = make_uint4(0, 0, 0, 0);
  if (UNEVEN && tid < 2) rooms[tid] = even;
  __syncthreads();
  const bool words = a.k % 64 == 0;                   // rows of scales start on 4 bytes
  const uint8_t* s[2] = {};                           // this thread's scales at k = 0
  int load_item = item_first, load_k0 = k_first, load_k = 0, load_row = 0;
  uint32_t scale[DEPTH][2][2] = {};                   // four scales a row, or two and two apart
  uint32_t phase = 0, used = 0, pending = 0;          // a bit a place
  bool ok = true;                                     // no wait of the warp ran out
  const int whole_to = words ? a.k - STEP_K : -1;     // a step from here has all its scales
  int load_end = 0;
  auto load_start = [&](int room) {
    load_k = start_of(load_k0);
    load_end = load_item < item_end ? min(load_k0 + room, k_end) : 0;
    if (load_item >= item_end) return;
    const Item item = item_at(load_item);
    const int n = item.n0 + tile * 16;
    load_row = item.e * a.n + item.n0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      s[h] = a.w_s + (static_cast<int64_t>(item.e) * a.n + min(n + g + 8 * h, a.n - 1)) * (a.k / 16) +
             4 * t;
  };
  auto load_next = [&](int i, uint32_t (&v)[2][2], int item) {
    if (ok && load_k < load_end) {
      if (tile == 0) {
        // The place has been read by all the part's warps.
        if (used >> i & 1) {
          ok = __all_sync(~0u, mbar_wait_bounded(empties + 8 * i, ~phase >> i & 1, a.timeout_ns));
        }
        if (ok && elect_one()) {
          mbar_arrive_expect_tx(fulls + 8 * i, tiles * STEP_BYTES);
          tma_load_2d(ring + i * (tiles * STEP_BYTES), &codes, load_k / 2, load_row, fulls + 8 * i);
        }
      }
      used |= 1u << i;
      pending |= 1u << i;
      if (load_k <= whole_to) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v[h][0] = __ldg(reinterpret_cast<const uint32_t*>(s[h] + load_k / 16));
          v[h][1] = 0;
        }
      } else {
        const int left = a.k - load_k - 64 * t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(s[h] + load_k / 16);
          const uint32_t lo = left > 0 ? __ldg(p) : 0, hi = left > 32 ? __ldg(p + 1) : 0;
          v[h][0] = lo;
          v[h][1] = hi;
        }
      }
    }
    load_k += turn;
    if (i == DEPTH - 1 && load_k >= load_end) {
      // The loads can be two short chunks ahead, and so have to leave one of an item
      // after this one's, whose expert's rows are not known yet.
      load_k0 += room_of(load_item != item);
      if (load_k0 >= k_end) {
        load_k0 = k_first;
        ++load_item;
      }
      load_start(room_of(load_item != item));
    }
  };
  auto wait_for = [&](int i) {
    ok = ok && __all_sync(~0u, mbar_wait_bounded(fulls + 8 * i, phase >> i & 1, a.timeout_ns));
    if (ok) {
      phase ^= 1u << i;
      pending &= ~(1u << i);
    }
    __syncwarp();
  };
  auto release = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(empties + 8 * i);
  };
  int held_item = -1, held_k0 = 0;                    // the chunk that they hold the start of

  // Up to `cap` rows of expert e from row `from` on: `found` of them, row_at(i);
  // next_row is then the next one after them.
  int found = 0, next_row = 0, row0 = 0;
  auto list_rows = [&](int e, int from) {
    if (!a.experts) {
      row0 = from;
      found = min(cap, a.rows - from);
      next_row = from + found;
      return;
    }
    __syncthreads();
    if (warp == 0) {
      int at = from, have = 0;
      bool past = false;
      while (at < a.rows && !past) {
        const int r = at + lane;
        const uint32_t hits = __ballot_sync(~0u, r < a.rows && a.experts[r] == e);
        const int place = have + __popc(hits & ((1u << lane) - 1)), free = cap - have;
        if ((hits >> lane & 1) && place < cap) list[place] = r;
        past = __popc(hits) > free;
        at += past ? static_cast<int>(__fns(hits, 0, free + 1)) : 32;
        have = min(have + __popc(hits), cap);
      }
      if (lane == 0) {
        list[TOKS] = have;
        list[TOKS + 1] = at;
        if constexpr (UNEVEN) {
          const int room = min(room_for(have), max(range, 1) * STEP_K);
          list[TOKS + 2] = from == 0 && rooms[1] != room;
          rooms[0] = room;
          if (from == 0) rooms[1] = room;
        }
      }
    }
    __syncthreads();
    found = list[TOKS];
    next_row = list[TOKS + 1];
    // What the loads hold was cut to the last expert's chunks.
    if (UNEVEN && list[TOKS + 2]) held_item = -1;
  };
  auto row_at = [&](int m) { return a.experts ? list[m] : row0 + m; };

  bool again = false;           // something is staged
  // Stages rows [0, rows) of the list from k0 to k1, each piece of 8 values
  // where the multiplication reads it: first as they are, then, when the rows'
  // largest magnitudes below `below` are known, the window from there down as
  // f16.  True where smaller ones are left.
  auto stage = [&](int rows, int k0, int k1, float global, int (&below)[TILES]) {
    const int all = (k1 - k0 + STEP_K - 1) / STEP_K * (STEP_K / 8);
    const int per = rows <= 1 ? 8 : rows <= 2 ? 4 : rows <= 4 ? 2 : 1;   // warps a row
    // A warp's 32 pieces in an order that spreads its stores over the banks.
    const int p0 = (warp % per) * 32 + lane % 4 * 8 + lane / 4;
    // Piece p is k = 8 p: of its 256, thread (p / 8) % 4's piece p % 8.
    auto place = [&](int m, int p) {
      return xs + (((p / 32 * 8 + p % 8) * rows + m) * 4 + p / 8 % 4) * 16;
    };
    if (again) __syncthreads();            // the last reads of what was staged before
    again = true;
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const int m = warp / per + i * WARPS;
      if (m >= rows) break;
      const uint32_t lim = below[i] << 7;
      const int row = row_at(m);
      const uint4* x = reinterpret_cast<const uint4*>(
          a.x + static_cast<int64_t>(a.share == 1 ? row : row / a.share) * a.ldx + k0);
      // The largest magnitude, and 0x7FFF + m for the smallest m > 0 (so that 0
      // is the largest of these as signed numbers), a pair of each.
      uint32_t most = 0, least = 0x7FFF7FFF;
#pragma unroll 1
      for (int p = p0; p < all; p += BATCH * per * 32) {
        uint4 v[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const int at = p + b * per * 32;
          v[b] = 8 * at < k1 - k0 ? __ldg(x + at) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const int at = p + b * per * 32;
          if (at >= all) break;
          sts128(place(m, at), v[b].x, v[b].y, v[b].z, v[b].w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t mag = word(v[b], j) & 0x7FFF7FFF;
            if (below[i] < 256) mag = in_window(mag, 0, lim);
            most = __vmaxu2(most, mag);
            least = __vmins2(least, mag + 0x7FFF7FFF);
          }
        }
      }
      most = __reduce_max_sync(~0u, max(most & 0xFFFF, most >> 16));
      least ^= 0x80008000;                 // m - 1, or 0xFFFF
      least = __reduce_min_sync(~0u, min(least & 0xFFFF, least >> 16));
      if (lane == 0) extent[i * WARPS + warp] = least << 16 | most;
    }
    __syncthreads();
    bool left = false;
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const int m = warp / per + i * WARPS;
      if (m >= rows) break;
      const uint32_t lim = below[i] << 7;
      const uint32_t own = lane < per ? extent[i * WARPS + warp / per * per + lane] : 0xFFFF0000;
      const uint32_t least = __reduce_min_sync(~0u, own >> 16);
      const int most = static_cast<int>(__reduce_max_sync(~0u, own & 0xFFFF));
      const int high = most >> 7;
      if (lane == 0) {                     // the same from each of the row's warps
        // G_e over the rows' factor; both in one step and the powers of two apart,
        // so that only a result out of fp32's range leaves it.
        int n;
        const float frac = frexpf(global, &n);
        n -= min(141 - high, 127);
        const int n1 = max(-125, min(n, 127)), n2 = max(-126, min(n - n1, 127));
        unit[m] = make_float2(frac * __int_as_float((n1 + 127) << 23),
                              __int_as_float((n2 + 127) << 23));
      }
      const uint32_t low = max(high - 28, 0) << 7;
      const float up = __uint_as_float(static_cast<uint32_t>(min(141 - high, 127) + 127) << 23);
      const bool some = least + 1 < low;   // smaller ones than the window's
      left |= some;
      const bool whole_row = !some && below[i] == 256;
#pragma unroll 1
      for (int p = p0; p < all; p += per * 32) {
        uint4 v = lds128(place(m, p));
        uint32_t o[4];
        if (!whole_row) {
          v.x = in_window(v.x, low, lim);
          v.y = in_window(v.y, low, lim);
          v.z = in_window(v.z, low, lim);
          v.w = in_window(v.w, low, lim);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          asm("cvt.rn.f16x2.f32 %0, %1, %2;"
              : "=r"(o[j]) : "f"(bf16_hi(word(v, j)) * up), "f"(bf16_lo(word(v, j)) * up));
        sts128(place(m, p), o[0], o[1], o[2], o[3]);
      }
      below[i] = max(high - 28, 0);
    }
    return __syncthreads_or(left) != 0;
  };

  // Adds the sums of `count` items from the first one on and writes them: a
  // thread a column, a pair of an item and a row at a time.
  auto flush = [&](int first, int count, int rows) {
    const int width = tiles * 16, col = tid % width, step = 32 * WARPS / width;
    __syncthreads();
    auto place = [&](int pair, int p) {
      const int n = rows == 1 ? pair : pair / rows, r = pair - n * rows;
      return red + ((n * WARPS + p * tiles + col / 16) * rows + r) * 16 + col % 16;
    };
    auto write = [&](int pair, float v) {
      const int n = rows == 1 ? pair : pair / rows, at = item_at(first + n).n0 + col;
      if (at < a.n) store_out(a, row_at(pair - n * rows), at, v);
    };
    if (cluster == 1 || parts > 1) {
#pragma unroll 1
      for (int pair = tid / width; pair < count * rows; pair += step) {
        float v = 0;
#pragma unroll 1
        for (int p = 0; p < parts; ++p) v += *place(pair, p);
        if (cluster == 1) write(pair, v);
        else *place(pair, 0) = v;           // this thread's own
      }
    }
    if (cluster == 1) {
      __syncthreads();
      return;
    }
    cluster_sync();
#pragma unroll 1
    for (int pair = tid / width * cluster + rank; pair < count * rows; pair += step * cluster) {
      const uint32_t at = smem_addr(place(pair, 0));
      float from[8], v = 0;
#pragma unroll
      for (int p = 0; p < 8; ++p) from[p] = p < cluster ? ld_cluster_f32(at, p) : 0.f;
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p < cluster) v += from[p];
      write(pair, v);
    }
    cluster_sync();
  };

  int cur = -1;                 // the expert whose rows are listed,
  bool whole = false;           // all of them,
  int staged = -1;              // and which start of K is staged (in one window)
  int first = item_first;       // the first item whose sums wait
  for (int item = item_first; item < item_end; ++item) {
    const Item here = item_at(item);
    if (here.e != cur || !whole) {
      if (item > first) flush(first, item - first, found);
      first = item;
      list_rows(here.e, 0);
      cur = here.e;
      whole = next_row >= a.rows;
      staged = -1;
    }
    const float global = a.w_global[here.e];
    while (true) {
      const int rows = found, after = next_row;
      const int room = room_of(0);
      float out[TILES][4] = {};
      for (int k0 = k_first; k0 < k_end; k0 += room) {
        const int k1 = min(k0 + room, k_end);
        int below[TILES];                          // exponents still to take (this warp's rows)
#pragma unroll
        for (int i = 0; i < TILES; ++i) below[i] = 256;
        bool more = staged != k0;
        for (int window = 0; window == 0 || more; ++window) {
          if (more) {
            more = stage(rows, k0, k1, global, below);
            staged = window == 0 && !more ? k0 : -1;
          }
          float sum[TILES][4] = {};
          // DEPTH steps at a time: each is multiplied and its place loaded again.
          // Where the places hold something else, the first round only loads.
          bool fill = item != held_item || k0 != held_k0;
          if (fill) {
#pragma unroll 1
            for (int i = 0; i < DEPTH; ++i)
              if (pending >> i & 1) {
                wait_for(i);
                release(i);
              }
            load_item = item;
            load_k0 = k0;
            load_start(room);
          }
          int k = start_of(k0);
          // This thread's pieces of x at k = k0.
          uint32_t x_first[TILES], x_step[TILES];
#pragma unroll
          for (int m = 0; m < TILES; ++m) {
            const bool has = g + 8 * m < rows;
            x_first[m] = has ? xs + ((g + 8 * m) * 4 + t) * 16 : smem_addr(zeros);
            x_step[m] = has ? rows * 64 : 0;
          }
          bool filled = false;
          do {
            filled = fill;
            // Sums of at most 512 terms at a time: the instruction cuts its sums off.
            float acc[2][TILES][4] = {};
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
              if (!fill && k < k1) {
                wait_for(i);
                const uint32_t four[2] = {scale[i][0][0] | scale[i][0][1] << 16,
                                          scale[i][1][0] | scale[i][1][1] << 16};
                uint32_t x_at[TILES];
#pragma unroll
                for (int m = 0; m < TILES; ++m) x_at[m] = x_first[m] + (k - k0) / 32 * x_step[m];
                multiply_step<TOKS>(acc, ring + (i * tiles + tile) * STEP_BYTES, four, x_at, x_step,
                                    g, t);
                release(i);
              }
              load_next(i, scale[i], item);
              if (!fill) k += turn;
            }
#pragma unroll
            for (int m = 0; m < TILES; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[m][i] += acc[0][m][i] + acc[1][m][i];
            fill = false;
          } while (filled || k < k1);
          held_item = k0 + room < k_end ? item : item + 1;     // what the loads have begun
          held_k0 = k0 + room < k_end ? k0 + room : k_first;
          // To the output's units.
#pragma unroll
          for (int m = 0; m < TILES; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * m + 2 * t + i % 2;
              if (r < rows) out[m][i] += sum[m][i] * unit[r].x * unit[r].y;
            }
        }
      }
#pragma unroll
      for (int m = 0; m < TILES; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * m + 2 * t + i % 2;
          if (r < rows)
            red[(((item - first) * WARPS + warp) * rows + r) * 16 + g + 8 * (i / 2)] = out[m][i];
        }
      const int places = SUM_BYTES / (WARPS * 16 * 4) / rows;    // for items
      if (after < a.rows || item + 1 - first == places || item + 1 == item_end) {
        flush(first, item + 1 - first, rows);
        first = item + 1;
      }
      if (after >= a.rows) break;
      // More rows than one pass takes: the weights again.
      list_rows(here.e, after);
      first = item;
      staged = -1;
    }
  }
  // Copies still in flight (after a wait that ran out) land before the memory is
  // given back.
#pragma unroll 1
  for (int i = 0; i < DEPTH; ++i)
    if (pending >> i & 1) mbar_wait_bounded(fulls + 8 * i, phase >> i & 1, a.timeout_ns);
  if (!ok && a.dev_err) atomicOr(a.dev_err, MXQ_DEVERR_TIMEOUT);
}

}  // namespace

// One or two rows: of the cuts into 1, 2, 4 or 8 tiles an item, 8, 4, 2 or 1
// parts of K, the one with the least estimated time.  Few parts mean few copies
// and sums an item, many items an even load: 28672 x 8192 weights, one row, 36,
// 33.7, 32.4 and 35.8 us with 8, 4, 2 and 1 tiles; 38912 x 8192, an item of 8 a
// CTA, 38, 39, 41 and 45.  K over clusters only where even one tile an item leaves
// SMs free.
//
// More rows: 8 tiles, and K over clusters of the size with the least estimated
// time, so that the staged rows are shared out too (4099 x 11008 weights, thirteen
// rows: 17.4 us over clusters of 8, 84 in one CTA, 34 in halves; 14336 x 4096, four
// rows: 18.1, 14.5 and 19.2 us over clusters of 1, 2 and 4).
GemvPlan gemv_plan(int64_t rows, int64_t n, int64_t k, int64_t experts, int num_sms) {
  // At most this many experts have rows, and then this many rows each.
  const int64_t slots = experts == 0 ? 1 : rows < experts ? rows : experts;
  const int64_t each = (rows + slots - 1) / slots;
  // With more than 4 rows an expert on average some have more than 8, and would read
  // their weights twice (7 experts with 52 rows, 16455 x 960: 35 us sixteen rows at a
  // time, 55 eight; 11 with 36, 4633 x 4608: 90 and 54).
  const int toks = each > (experts > 0 ? 4 : 8) ? 16 : 8;
  const int x_bytes = toks == 16 ? Shape<16>::X_BYTES : Shape<8>::X_BYTES;
  const int64_t steps = (k + STEP_K - 1) / STEP_K;
  auto items = [&](int tiles) { return (n + tiles * 16 - 1) / (tiles * 16) * slots; };
  GemvPlan plan{toks, WARPS, 1, experts > 0 || rows > toks ? toks : static_cast<int>(rows), false};
  // Quarters of a round of two CTAs an SM; a last one of at most a CTA an SM takes
  // three.
  auto rounds = [&](int64_t n) {
    const int64_t rest = n % (2 * num_sms);
    return n / (2 * num_sms) * 4 + (rest > num_sms ? 4 : rest > 0 ? 3 : 0);
  };
  if (each <= 2) {
    // In eighths of a step of all warps, a step more an item.
    auto cost = [&](int tiles) { return rounds(items(tiles)) * (steps * tiles + 8); };
    for (int tiles = WARPS / 2; tiles > 0; tiles /= 2)
      if (cost(tiles) < cost(plan.tiles)) plan.tiles = tiles;
    while (plan.tiles == 1 && plan.cluster < 8 && items(1) * plan.cluster < num_sms * 3 / 2 &&
           steps >= 2 * WARPS * plan.cluster)
      plan.cluster *= 2;
  } else {
    // Staging and the sums over a cluster are worth four steps.
    auto cost = [&](int cluster) {
      return rounds(items(WARPS) * cluster) * (8 * steps / cluster + 32);
    };
    for (int cluster = 2; cluster <= 8 && cluster <= steps; cluster *= 2)
      if (cost(cluster) <= cost(plan.cluster)) plan.cluster = cluster;
  }
  while (plan.tiles > 1 && items(plan.tiles) * plan.cluster < num_sms / 2) plan.tiles /= 2;
  // Rows whose range of K is staged whole.  An expert with more than `cap` has its
  // weights read again, and how many one has is not known here: where a quarter of
  // the kernel's rows would be lost, the room follows each expert's rows instead (128
  // rows over 64 experts, 4096 x 7168, where 2 fit: 440 us two at a time, 210 so).
  // That costs ordinary calls a little (32 rows over 64 experts, 2816 x 2048, 7 fit:
  // 25.3 us seven at a time, 25.9 so).
  const int64_t range = (steps + plan.cluster - 1) / plan.cluster;
  const int64_t fit = x_bytes / (2 * STEP_K) / (range > 0 ? range : 1);
  if (experts > 0 && fit < toks) {
    plan.uneven = 4 * fit < 3 * toks;
    if (!plan.uneven) plan.cap = static_cast<int>(fit);
  }
  plan.items = items(plan.tiles);
  const int64_t most = 2 * num_sms / plan.cluster;
  plan.grid = static_cast<int>(plan.items < most ? plan.items : most) * plan.cluster;
  return plan;
}

namespace {

template <int TOKS, bool UNEVEN>
cudaError_t launch(const GemvArgs& a, const GemvPlan& plan, cudaStream_t stream) {
  constexpr int smem = Shape<TOKS>::SMEM;
  static std::atomic<uint64_t> allowed{0};
  auto kernel = nvfp4_gemv_kernel<TOKS, UNEVEN>;
  const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), smem, &allowed);
  if (e != cudaSuccess) return e;
  // w_q as rows of bytes, a copy of a line each of a CTA's rows.
  CUtensorMap codes{};
  if (a.k > 0) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.k / 2),
                                static_cast<cuuint64_t>(a.num_experts) * a.n};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.k / 2)};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(16 * plan.tiles)};
    if (encode_map(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.w_q, dims, strides, box,
                   CU_TENSOR_MAP_SWIZZLE_128B) != MXQ_OK)
      return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.grid));
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = plan.cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, codes, a, plan.tiles, plan.cluster, plan.cap);
}

}  // namespace

cudaError_t launch_nvfp4_gemv(const GemvArgs& a, const GemvPlan& plan, cudaStream_t stream) {
  if (plan.uneven)
    return plan.toks == 16 ? launch<16, true>(a, plan, stream) : launch<8, true>(a, plan, stream);
  return plan.toks == 16 ? launch<16, false>(a, plan, stream) : launch<8, false>(a, plan, stream);
}

}  // namespace mxq
