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
constexpr int BLOCK_K = 256;   // K of one prefetch step of a warp: 2 x 16 bytes of codes a row
constexpr int X_BYTES = 96 * 1024;   // staged rows of x: two CTAs share an SM

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

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The codes and scales that one thread multiplies in a step: of two rows, two
// pieces of 32 values (16 bytes of codes, two block scales).
struct Step {
  uint4 c[2][2];
  uint32_t s[2][2];
};

__device__ __forceinline__ void load_step(Step& w, const uint8_t* const (&q)[2],
                                          const uint8_t* const (&s)[2], int k, int limit) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = k + 128 * j;
      w.c[j][h] = make_uint4(0, 0, 0, 0);
      w.s[j][h] = 0;
      if (at < limit) {
        w.c[j][h] = __ldg(reinterpret_cast<const uint4*>(q[h] + at / 2));
        w.s[j][h] = __ldg(reinterpret_cast<const uint16_t*>(s[h] + at / 16));
      }
    }
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// One step: x fragments from shared memory at xs, 4 pieces of [rows][4] 16-byte
// units for each 128 of K.  Thread (g, t) holds weight rows g and g + 8, and
// row g (and g + 8) of x, at the 32 values of k that its codes stand for; the
// instruction's k order is the codes' order, on both sides.
template <int TOKS>
__device__ __forceinline__ void multiply_step(float (&acc)[TOKS / 8][4], const Step& w,
                                              uint32_t xs, int rows, int g, int t) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t sc[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t s2 = e4m3x2_to_f16(w.s[j][h]);
      sc[h][0] = prmt(s2, s2, 0x1010);
      sc[h][1] = prmt(s2, s2, 0x3232);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 x[TOKS / 8];
#pragma unroll
      for (int m = 0; m < TOKS / 8; ++m) {
        x[m] = make_uint4(0, 0, 0, 0);
        if (g + 8 * m < rows)
          x[m] = lds128(xs + (((j * 4 + i) * rows + g + 8 * m) * 4 + t) * 16);
      }
      uint32_t v[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        e2m1x8_to_f16(word(w.c[j][h], i), v[h]);
#pragma unroll
        for (int p = 0; p < 4; ++p) v[h][p] = mul_f16x2(v[h][p], sc[h][i / 2]);
      }
#pragma unroll
      for (int m = 0; m < TOKS / 8; ++m) {
        mma_f16(acc[m], v[0][0], v[1][0], v[0][1], v[1][1], x[m].x, x[m].y);
        mma_f16(acc[m], v[0][2], v[1][2], v[0][3], v[1][3], x[m].z, x[m].w);
      }
    }
  }
}

// A CTA multiplies 16 * tiles weight rows by up to TOKS rows of x over its part
// of K; its 8 warps are `tiles` row tiles x 8 / tiles parts of K (taken step
// by step in turn).  The parts' sums are added through shared memory, and
// those of a cluster's CTAs through the first one's, in a fixed order.
template <int TOKS>
__global__ void __launch_bounds__(32 * WARPS, 2)
nvfp4_gemv_kernel(const GemvArgs a, const int tiles, const int cluster, const int by_row) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_up_shared<16>(smem_raw);
  float* red = reinterpret_cast<float*>(smem);            // [warp][16][TOKS]
  const uint32_t xs = smem_addr(smem + WARPS * 16 * TOKS * 4);
  __shared__ int list[TOKS];
  __shared__ int found, next_row;
  __shared__ int top[TOKS];                               // largest magnitude left of each row
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int rank = blockIdx.x % cluster, n0 = blockIdx.x / cluster * tiles * 16;
  const int cols = min(tiles * 16, a.n - n0);

  // This CTA's expert.  by_row: the one of row blockIdx.y, unless an earlier
  // row has it already.
  int e = blockIdx.y, from = 0;
  if (by_row) {
    from = blockIdx.y;
    e = a.experts[from];
    bool mine = true;
    for (int i = tid; i < from; i += 32 * WARPS) mine &= a.experts[i] != e;
    if (e < 0 || e >= a.num_experts) {
      for (int i = tid; rank == 0 && i < cols; i += 32 * WARPS) store_out(a, from, n0 + i, 0.f);
      return;
    }
    if (!__syncthreads_and(mine)) return;
  } else if (a.experts && blockIdx.y == 0 && rank == 0) {
    for (int r = 0; r < a.rows; ++r) {
      const int id = a.experts[r];
      if (id < 0 || id >= a.num_experts)
        for (int i = tid; i < cols; i += 32 * WARPS) store_out(a, r, n0 + i, 0.f);
    }
  }

  // This warp's weight rows and steps.
  const int parts = WARPS / tiles, tile = warp % tiles, part = warp / tiles;
  const uint8_t *q[2], *s[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t n = static_cast<int64_t>(e) * a.n + min(n0 + tile * 16 + g + 8 * h, a.n - 1);
    q[h] = a.w_q + n * (a.k / 2);
    s[h] = a.w_s + n * (a.k / 16);
  }
  const int steps = (a.k + BLOCK_K - 1) / BLOCK_K, share = (steps + cluster - 1) / cluster;
  const int k_first = min(rank * share, steps) * BLOCK_K;
  const int k_end = min(min((rank + 1) * share, steps) * BLOCK_K, a.k);
  int exp_g;
  const float frac_g = frexpf(a.w_global[e], &exp_g);
  Step w;
  load_step(w, q, s, k_first + part * BLOCK_K + 32 * t, k_end);   // before x is known

  if (tid == 0) next_row = from;
  __syncthreads();
  while (next_row < a.rows) {
    // Up to TOKS rows of this expert.
    __syncthreads();
    if (warp == 0) {
      int at = next_row, have = 0;
      while (at < a.rows && have < TOKS) {
        const int r = at + lane;
        const bool hit = r < a.rows && (!a.experts || a.experts[r] == e);
        const uint32_t hits = __ballot_sync(~0u, hit);
        const int place = have + __popc(hits & ((1u << lane) - 1));
        if (hit && place < TOKS) list[place] = r;
        const int room = TOKS - have;
        if (__popc(hits) > room) {      // the row after the last one taken
          at += __fns(hits, 0, room + 1);
          have = TOKS;
        } else {
          at += 32;
          have += __popc(hits);
        }
      }
      if (lane == 0) {
        found = have;
        next_row = at;
      }
    }
    __syncthreads();
    const int rows = found;
    if (rows == 0) break;

    float out[TOKS / 8][4] = {};
    const int room_k = X_BYTES / (rows * 2) / BLOCK_K * BLOCK_K;
    for (int k0 = k_first; k0 < k_end; k0 += room_k) {
      const int k1 = min(k0 + room_k, k_end);
      const int pieces = (k1 - k0) / 8;          // 16-byte pieces of a row of x
      const int per = rows <= 1 ? 8 : rows <= 2 ? 4 : rows <= 4 ? 2 : 1;   // warps a row
      int below = 256;                           // exponents still to take (this warp's rows)
      int below2 = 256;
      bool more = true;
      while (more) {
        if (tid < TOKS) top[tid] = 0;
        __syncthreads();
        for (int m = warp / per; m < rows; m += WARPS / per) {
          const uint16_t* x = a.x + static_cast<int64_t>(list[m] / a.share) * a.ldx + k0;
          const uint32_t lim = (m < WARPS / per ? below : below2) << 7;
          uint32_t best = 0;
          for (int p = (warp % per) * 32 + lane; p < pieces; p += per * 32) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(x) + p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t lo = word(v, i) & 0x7FFF, hi = (word(v, i) >> 16) & 0x7FFF;
              if (lo < lim) best = max(best, lo);
              if (hi < lim) best = max(best, hi);
            }
          }
          best = __reduce_max_sync(~0u, best);
          if (lane == 0) atomicMax(&top[m], static_cast<int>(best));
        }
        __syncthreads();
        bool left = false;
        for (int m = warp / per; m < rows; m += WARPS / per) {
          const uint16_t* x = a.x + static_cast<int64_t>(list[m] / a.share) * a.ldx + k0;
          int& mine = m < WARPS / per ? below : below2;
          const uint32_t lim = mine << 7;
          const int high = top[m] >> 7;
          const uint32_t low = max(high - 28, 0) << 7;
          const float up = __uint_as_float(static_cast<uint32_t>(min(141 - high, 127) + 127) << 23);
          for (int p = (warp % per) * 32 + lane; p < (k1 - k0 + BLOCK_K - 1) / BLOCK_K * (BLOCK_K / 8);
               p += per * 32) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (p < pieces) v = __ldg(reinterpret_cast<const uint4*>(x) + p);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t lo = word(v, i) & 0x7FFF, hi = (word(v, i) >> 16) & 0x7FFF;
              left |= (lo < low && lo != 0) || (hi < low && hi != 0);
              const float f0 = lo >= low && lo < lim ? bf16_lo(word(v, i)) * up : 0.f;
              const float f1 = hi >= low && hi < lim ? bf16_hi(word(v, i)) * up : 0.f;
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(f1), "f"(f0));
            }
            // Piece p is k = 8 p: of its 128, thread t = (p / 4) % 4's piece p % 4.
            sts128(xs + (((p / 16 * 4 + p % 4) * rows + m) * 4 + p / 4 % 4) * 16, o[0], o[1], o[2],
                   o[3]);
          }
          mine = max(high - 28, 0);
        }
        more = __syncthreads_or(left);

        float sum[TOKS / 8][4] = {};
        for (int k = k0 + part * BLOCK_K; k < k1; k += parts * BLOCK_K) {
          Step now = w;
          int ahead = k + parts * BLOCK_K;
          if (ahead >= k1) ahead = (more ? k0 : k1) + part * BLOCK_K;
          load_step(w, q, s, ahead + 32 * t, k_end);
          // Sums of 256 terms at a time: the instruction cuts its sums off.
          float acc[TOKS / 8][4] = {};
          multiply_step<TOKS>(acc, now, xs + (k - k0) * rows * 2, rows, g, t);
#pragma unroll
          for (int m = 0; m < TOKS / 8; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[m][i] += acc[m][i];
        }
        // To the output's units; both scales in one step, so that only a
        // result out of fp32's range leaves it.
#pragma unroll
        for (int m = 0; m < TOKS / 8; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * m + 2 * t + i % 2;
            const int high = r < rows ? top[r] >> 7 : 0;
            out[m][i] += ldexpf(sum[m][i] * frac_g, exp_g - min(141 - high, 127));
          }
        __syncthreads();
      }
    }

    // Sums of this CTA's parts of K, then of the cluster's.
#pragma unroll
    for (int m = 0; m < TOKS / 8; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(warp * TOKS + 8 * m + 2 * t + i % 2) * 16 + g + 8 * (i / 2)] = out[m][i];
    __syncthreads();
    for (int i = tid; i < tiles * 16 * rows; i += 32 * WARPS) {
      const int col = i % (tiles * 16), r = i / (tiles * 16);
      float v = 0;
      for (int p = 0; p < parts; ++p)
        v += red[((p * tiles + col / 16) * TOKS + r) * 16 + col % 16];
      if (cluster == 1) {
        if (col < cols) store_out(a, list[r], n0 + col, v);
      } else {
        red[((col / 16) * TOKS + r) * 16 + col % 16] = v;   // part 0's place, this thread's own
      }
    }
    if (cluster > 1) {
      cluster_sync();
      for (int i = tid; rank == 0 && i < cols * rows; i += 32 * WARPS) {
        const int col = i % cols, r = i / cols;
        const uint32_t at = smem_addr(red + ((col / 16) * TOKS + r) * 16 + col % 16);
        float v = 0;
        for (int p = 0; p < cluster; ++p) v += ld_cluster_f32(at, p);
        store_out(a, list[r], n0 + col, v);
      }
      cluster_sync();
    }
    // More rows than one pass takes: the weights again from the start.
    if (next_row < a.rows) load_step(w, q, s, k_first + part * BLOCK_K + 32 * t, k_end);
    __syncthreads();
  }
}

template <int TOKS>
cudaError_t launch(const GemvArgs& a, int tiles, int cluster, int slots, bool by_row,
                   cudaStream_t stream) {
  constexpr int smem = X_BYTES + WARPS * 16 * TOKS * 4 + 16;
  cudaError_t e = cudaFuncSetAttribute(nvfp4_gemv_kernel<TOKS>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int groups = (a.n + tiles * 16 - 1) / (tiles * 16);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(groups) * cluster, slots);
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, nvfp4_gemv_kernel<TOKS>, a, tiles, cluster, by_row ? 1 : 0);
}

}  // namespace

cudaError_t launch_nvfp4_gemv(const GemvArgs& a, int num_sms, cudaStream_t stream) {
  // A grid row for each expert, or for each row where there are fewer rows.
  const bool by_row = a.experts && a.rows <= a.num_experts && a.rows <= 65535;
  const int slots = !a.experts ? 1 : by_row ? a.rows : a.num_experts;
  // Rows that a CTA is likely to multiply at once.
  const int rows = a.experts ? (a.rows + a.num_experts - 1) / a.num_experts : a.rows;
  const int steps = (a.k + BLOCK_K - 1) / BLOCK_K;
  // Enough CTAs for two on every SM, with the fewest parts of K.
  const int64_t row_tiles = (static_cast<int64_t>(a.n) + 15) / 16;
  int tiles = 8, cluster = 1;
  while (tiles > 1 && (row_tiles + tiles - 1) / tiles * slots < 2 * num_sms) tiles /= 2;
  while (cluster < 8 && (row_tiles + tiles - 1) / tiles * slots * cluster < num_sms &&
         steps > 2 * cluster * (WARPS / tiles))
    cluster *= 2;
  return rows > 8 ? launch<16>(a, tiles, cluster, slots, by_row, stream)
                  : launch<8>(a, tiles, cluster, slots, by_row, stream);
}

}  // namespace mxq
