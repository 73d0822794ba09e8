// moe_kernels.cu -- routing of tokens to experts, its backward pass, and the
// sorting of (token, expert) pairs into the rows of the grouped products.
//
// Routing: one warp a token, VPL neighbouring experts a lane.  Each lane sorts its
// keys by a network of minima and maxima; the k best of the warp then come out one
// after another, each the largest of the lanes' heads (one reduction across the warp,
// and the lowest lane that has it).  Which expert a key is of is looked up once for
// all slots.  Keys are computed in 32 bits with a known error; where two that decide
// about an expert or about the order are nearer than their errors, the experts near
// the border are compared again in 64 bits, so that the choice is that of the exact
// scores.  That happens to about one token in a thousand.

#include <cooperative_groups.h>
#include <cfloat>

#include "mxq_internal.h"
#include "mxq_layer.h"
#include "mxq_products.h"
#include "mxq_ptx.cuh"

namespace mxq {
namespace {

namespace cg = cooperative_groups;

constexpr uint32_t FULL = 0xFFFFFFFFu;
constexpr int ROUTE_WARPS = 4;
// CTAs of 128 threads an SM: 64 registers a thread, of which a few spill from twelve
// experts a lane on (16384 tokens, 8 of 512 with a bias: 25.1 us, with 80 registers 26.4; 8
// of 384 17.4 and 18.4).
constexpr int ROUTE_CTAS = 8;

__device__ __forceinline__ float infinity() { return __int_as_float(0x7F800000); }

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) {
  uint16_t b;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
  *p = b;
}

// Largest value of the warp's lanes, none of them NaN.
__device__ __forceinline__ float redux_max(float v) {
  float d;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float LOG2E = 1.4426950408889634f;

// Sorts v[0 .. N) in descending order (Batcher's odd-even merge network).
template <int N>
__device__ __forceinline__ void sort_descending(float (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const float a = v[i + j], b = v[i + j + k];
            v[i + j] = fmaxf(a, b);
            v[i + j + k] = fminf(a, b);
          }
}

// Bytes of the widest access that N values of SIZE bytes are a whole number of.
template <int N, int SIZE>
constexpr int access_bytes() {
  return N * SIZE % 16 == 0 ? 16 : N * SIZE % 8 == 0 ? 8 : N * SIZE % 4 == 0 ? 4 : 2;
}

// N values of type float or bf16 from p, in accesses of access_bytes() where `wide` says
// that they start on a multiple of that.
template <int N>
__device__ __forceinline__ void load_values(const float* p, bool wide, float (&v)[N]) {
  if (wide && N % 4 == 0) {
#pragma unroll
    for (int i = 0; i + 3 < N; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  } else if (wide && N % 2 == 0) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
      const float2 x = *reinterpret_cast<const float2*>(p + i);
      v[i] = x.x;
      v[i + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i];
  }
}
template <int N>
__device__ __forceinline__ void load_values(const uint16_t* p, bool wide, float (&v)[N]) {
  if (wide && N >= 2) {
    uint32_t w[(N + 1) / 2];
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N / 2; i += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + 2 * i);
        w[i] = x.x;
        w[i + 1] = x.y;
        w[i + 2] = x.z;
        w[i + 3] = x.w;
      }
    } else if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N / 2; i += 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p + 2 * i);
        w[i] = x.x;
        w[i + 1] = x.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = load_logit(p + i);
  }
}

template <typename T>
__device__ __forceinline__ T warp_max(T v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const T o = __shfl_xor_sync(FULL, v, d);
    v = o > v ? o : v;
  }
  return v;
}
template <typename T>
__device__ __forceinline__ T warp_add(T v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
  return v;
}

// The sigmoid's two factors: sigmoid(l) = n e^min(l, 0) with n = 1 / (1 + e^-|l|).
__device__ __forceinline__ float sigmoid_n(float l) {
  return __fdividef(1.0f, 1.0f + expf(-fabsf(l)));      // the divisor is between 1 and 2
}
__device__ __forceinline__ float sigmoid_of(float l) {
  const float n = sigmoid_n(l);
  return l >= 0.0f ? n : n * expf(l);
}

// The two largest of two pairs.
template <typename T>
__device__ __forceinline__ void merge_two(T& a1, T& a2, T b1, T b2) {
  const T low = a1 < b1 ? a1 : b1, second = a2 > b2 ? a2 : b2;
  a1 = a1 < b1 ? b1 : a1;
  a2 = low > second ? low : second;
}

// expert / size for expert < 512: recip = ceil(2^32 / size), or 0 for size 1.
__device__ __forceinline__ int group_of(int e, uint32_t recip) {
  return recip == 0u ? e : static_cast<int>(__umulhi(static_cast<uint32_t>(e), recip));
}

template <int N>
__device__ __forceinline__ void store_values(float* p, const float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) *reinterpret_cast<float2*>(p + i) = make_float2(v[i], v[i + 1]);
  } else {
    *p = v[0];
  }
}

struct Choice {
  RouteArgs a;
  int group_size;
  uint32_t recip;
  int spread;               // log2 of the lanes a group, of 32 / (groups rounded up to 2^n)
  int own;                  // log2 of the lanes that hold a group's experts and no others, or -1
  int wide;                 // bits: a lane's logits, its biases are aligned
};

// Which groups are kept, as bits g << spread, from the lanes g << spread .. holding
// group g's score.
__device__ __forceinline__ uint32_t keep_groups(double score, int groups, int kept, int spread,
                                                int lane) {
  const int g = lane >> spread;
  int rank = 0;
  for (int o = 0; o < groups; ++o) {
    const double s = __shfl_sync(FULL, score, o << spread);
    rank += s > score || (s == score && o < g);
  }
  return __ballot_sync(FULL, g < groups && lane == g << spread && rank < kept);
}

// The choice in 64 bits: slot i's expert in lane i (-1 where there is none).
template <int VPL>
__device__ __forceinline__ int choose_exactly(const Choice& ch, const float* logits, float top) {
  const RouteArgs& a = ch.a;
  const int lane = threadIdx.x & 31;
  const double none = -static_cast<double>(infinity());
  const bool sigmoid = (a.flags & MXQ_ROUTE_SIGMOID) != 0;
  double total = 0.0;
  if (!sigmoid) {
    for (int e = lane; e < a.experts; e += 32)
      total += exp(static_cast<double>(logits[e]) - static_cast<double>(top));
    total = warp_add(total);
  }
  double key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = 32 * j + lane;
    key[j] = none;
    if (e >= a.experts || !(logits[e] > -infinity())) continue;
    const double l = logits[e];
    const double s = sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - static_cast<double>(top)) / total;
    key[j] = a.bias ? s + static_cast<double>(a.bias[e]) : s;
  }
  if (a.groups > 1) {
    double mine = none;
    for (int g = 0; g < a.groups; ++g) {
      double t1 = none, t2 = none;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (32 * j + lane < a.experts && group_of(32 * j + lane, ch.recip) == g)
          merge_two(t1, t2, key[j], none);
      for (int d = 16; d >= 1; d >>= 1) {
        const double o1 = __shfl_xor_sync(FULL, t1, d), o2 = __shfl_xor_sync(FULL, t2, d);
        merge_two(t1, t2, o1, o2);
      }
      const double s = (a.flags & MXQ_ROUTE_GROUP_MAX) || ch.group_size == 1 ? t1 : t1 + t2;
      if (lane >> ch.spread == g) mine = s;
    }
    const uint32_t keep = keep_groups(mine, a.groups, a.kept, ch.spread, lane);
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (!(keep >> (group_of(32 * j + lane, ch.recip) << ch.spread & 31) & 1u)) key[j] = none;
  }
  if (!a.bias) {
    // Without a bias the logits' own order: scores may coincide where they differ.
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] > none) key[j] = logits[32 * j + lane];
  }
  int chosen = -1;
  for (int r = 0; r < a.slots; ++r) {
    double best = none;
    int at = 1 << 20;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] > best) {
        best = key[j];
        at = 32 * j + lane;
      }
    for (int d = 16; d >= 1; d >>= 1) {
      const double o = __shfl_xor_sync(FULL, best, d);
      const int oa = __shfl_xor_sync(FULL, at, d);
      if (o > best || (o == best && oa < at)) {
        best = o;
        at = oa;
      }
    }
    if (!(best > none)) break;
    if (lane == r) chosen = at;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (32 * j + lane == at) key[j] = none;
  }
  return chosen;
}

// An expert's key in 64 bits; `total` is the softmax's sum.
__device__ __forceinline__ double key64(const RouteArgs& a, const float* logits, int e, float top,
                                        double total) {
  const double l = logits[e];
  const double s = (a.flags & MXQ_ROUTE_SIGMOID) ? 1.0 / (1.0 + exp(-l))
                                                 : exp(l - static_cast<double>(top)) / total;
  return a.bias ? s + static_cast<double>(a.bias[e]) : s;
}

__device__ __forceinline__ double total64(const RouteArgs& a, const float* logits, float top) {
  if (a.flags & MXQ_ROUTE_SIGMOID) return 1.0;
  double total = 0.0;
  // (Rolled: code that few tokens reach is fetched when they do, and takes registers.)
#pragma unroll 1
  for (int e = threadIdx.x & 31; e < a.experts; e += 32)
    total += exp(static_cast<double>(logits[e]) - static_cast<double>(top));
  return warp_add(total);
}

// The choice among the experts e of the lanes 0 .. n - 1 by keys in 64 bits: slot i's
// expert in lane i.
__device__ __forceinline__ int choose_near(const RouteArgs& a, const float* logits, float top, int e,
                                        int n) {
  const int lane = threadIdx.x & 31;
  const double total = total64(a, logits, top);
  const double key = lane < n ? key64(a, logits, e, top, total) : 0.0;
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const double k = __shfl_sync(FULL, key, i);
    const int o = __shfl_sync(FULL, e, i);
    rank += k > key || (k == key && o < e);
  }
  int chosen = -1;
  for (int i = 0; i < n; ++i) {
    const int r = __shfl_sync(FULL, rank, i), o = __shfl_sync(FULL, e, i);
    if (r == lane) chosen = o;
  }
  return lane < a.slots ? chosen : -1;
}

// The kept groups (bits g << spread) by scores in 64 bits of the experts e of the lanes
// 0 .. n - 1, which hold every group's two best.
__device__ __forceinline__ uint32_t keep_near(const Choice& ch, const float* logits, float top, int e,
                                           int n, int spread) {
  const RouteArgs& a = ch.a;
  const int lane = threadIdx.x & 31;
  const double none = -static_cast<double>(infinity());
  const double total = total64(a, logits, top);
  const double key = lane < n ? key64(a, logits, e, top, total) : none;
  const int group = lane < n ? group_of(e, ch.recip) : -1;
  double t1 = none, t2 = none;
  for (int i = 0; i < n; ++i) {
    const double k = __shfl_sync(FULL, key, i);
    if (__shfl_sync(FULL, group, i) == lane >> spread) merge_two(t1, t2, k, none);
  }
  const double s = (a.flags & MXQ_ROUTE_GROUP_MAX) || ch.group_size == 1 ? t1 : t1 + t2;
  return keep_groups(s, a.groups, a.kept, spread, lane);
}

template <typename T, int VPL>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, ROUTE_CTAS) moe_route_kernel(const Choice ch) {
  const RouteArgs& a = ch.a;
  constexpr int SPAN = 32 * VPL;
  __shared__ __align__(16) float s_logits[ROUTE_WARPS][SPAN];
  __shared__ __align__(16) float s_keys[ROUTE_WARPS][SPAN];
  __shared__ float s_queue[ROUTE_WARPS][SPAN + 32];     // [place][lane], and -inf
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + warp;
  if (token >= a.tokens) return;
  const bool sigmoid = (a.flags & MXQ_ROUTE_SIGMOID) != 0;
  const bool renorm = (a.flags & MXQ_ROUTE_RENORM) != 0;
  const bool grouped = a.groups > 1 && a.kept < a.groups;
  const T* row = static_cast<const T*>(a.logits) + token * a.ldl;
  float* sl = s_logits[warp];
  const float none = -infinity();
  const int e0 = lane * VPL;                          // this lane's experts e0 .. e0 + VPL - 1

  float l[VPL];
  if (e0 + VPL <= a.experts) {
    load_values<VPL>(row + e0, ch.wide & 1, l);
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) l[j] = e0 + j < a.experts ? load_logit(row + e0 + j) : none;
  }
  float most = l[0];
#pragma unroll
  for (int j = 1; j < VPL; ++j) most = max_nan(most, l[j]);
  int32_t* ids = a.ids + token * a.slots;
  float* weights = a.weights + token * a.slots;
  if (__any_sync(FULL, !(most < infinity()))) {       // NaN or +inf
    if (lane < a.slots) {
      ids[lane] = -1;
      weights[lane] = __int_as_float(0x7FC00000);
    }
    return;
  }
  store_values(sl + e0, l);

  // The softmax's largest logit and sum, where scores are needed.
  float top = 0.0f, total = 1.0f, inv = 1.0f;
  if (!sigmoid && (a.bias || grouped || !renorm)) {
    top = redux_max(most);
    if (!(top > none)) top = 0.0f;
    total = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) total += ex2_fast((l[j] - top) * LOG2E);
    total = warp_add(total);
    inv = total > 0.0f ? rcp_fast(total) : 0.0f;
  }
  // (Explicit roundings: the same logit and bias have the same key in every lane, which
  // products and sums that the compiler fuses here and not there would not keep.)
  auto score = [&](float x) {
    return sigmoid ? rcp_fast(__fadd_rn(1.0f, ex2_fast(__fmul_rn(-x, LOG2E))))
                   : __fmul_rn(ex2_fast(__fmul_rn(__fadd_rn(x, -top), LOG2E)), inv);
  };
  // What a score is off by at most.  Sigmoid, its slope at most 1/4 and |l| times that
  // at most 0.23: 2^-22 for e^-l, |l| 1.5 2^-24 for its argument, a rounding and 2^-23
  // for the quotient.  Softmax, in units of the largest score `inv`: two exponentials
  // at 2^-22, |l - top| e^(l - top) 2.5 2^-24 for their arguments, 21 additions, and
  // the quotient: 2.1e-6.
  const float err = sigmoid ? 4e-7f : 2.5e-6f * inv;

  float key[VPL];
  if (a.bias) {
    float b[VPL];
    if (e0 + VPL <= a.experts) {
      load_values<VPL>(a.bias + e0, ch.wide & 2, b);
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) b[j] = e0 + j < a.experts ? a.bias[e0 + j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = l[j] > none ? __fadd_rn(score(l[j]), b[j]) : none;
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = l[j] + 0.0f;      // -0 is 0
  }
  // Without a bias the keys are the logits.
  float* sk = a.bias ? s_keys[warp] : sl;
  if (a.bias) store_values(sk + e0, key);
  __syncwarp();

  bool unsure = false;          // 64 bits for all experts
  // Which groups are kept (bits g << spread), from the two largest keys of each lane that
  // has a part of group lane >> spread.
  auto group_kept = [&](float t1, float t2, int spread) -> uint32_t {
    for (int d = 1; d < 1 << spread; d <<= 1) {
      const float o1 = __shfl_xor_sync(FULL, t1, d), o2 = __shfl_xor_sync(FULL, t2, d);
      merge_two(t1, t2, o1, o2);
    }
    const float second = t2;
    if (!a.bias) {              // keys are logits
      t1 = t1 > none ? score(t1) : none;
      t2 = t2 > none ? score(t2) : none;
    }
    const int g = lane >> spread;
    const bool in = g < a.groups;
    const bool alone = (a.flags & MXQ_ROUTE_GROUP_MAX) || ch.group_size == 1;
    // (The mean of the two: their sum may pass fp32's range.)
    const float s = 0.5f * t1 + 0.5f * (alone ? t1 : t2);
    // The best group a.kept times, and the next one's score; equal groups in order.
    uint32_t keep = 0u;
    float rest = in ? s : none, worst = none;
    bool left = in;
    for (int i = 0; i < a.kept; ++i) {
      worst = redux_max(left ? rest : none);
      const int first = __ffs(__ballot_sync(FULL, left && rest == worst)) - 1;
      keep |= 1u << first;
      left = left && g != first >> spread;
    }
    const float next = redux_max(left ? rest : none);
    // The mean of two scores a side, each off by err and, with its bias, a rounding, and the
    // rounding of their sum.  Groups at -inf are behind the others, and a tie.
    const float amp = redux_max((t1 > none ? fabsf(t1) : 0.0f) + (t2 > none ? fabsf(t2) : 0.0f));
    if (!(next > none && worst - next <= 2.0f * err + 1.2e-7f * amp)) return keep;
    // Every expert that may be one of its group's two best, a lane each: logits have
    // their own order, keys are off by err and a rounding.
    const float slack = a.bias ? 2.0f * err + 2.4e-7f * (fabsf(second) + 1.0f) : 0.0f;
    int n = 0, mine = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const float k = sk[e0 + j];
      const float border = __shfl_sync(FULL, second - slack, group_of(e0 + j, ch.recip) << spread & 31);
      const bool may = k > none && (k >= border || !(border > none));
      uint32_t all = __ballot_sync(FULL, may);
      // The lane that becomes number n + i of the list is lane n + i.
      for (; all != 0u && n < 33; all &= all - 1u, ++n)
        if (lane == n) mine = (__ffs(all) - 1) * VPL + j;
    }
    if (n > 32) {
      unsure = true;
      return keep;
    }
    return keep_near(ch, sl, top, mine, n, spread);
  };
  if (grouped && ch.own < 0) {
    float t1 = none, t2 = none;
    const int g = lane >> ch.spread;
    if (g < a.groups)
      for (int i = lane & ((1 << ch.spread) - 1); i < ch.group_size; i += 1 << ch.spread)
        merge_two(t1, t2, sk[g * ch.group_size + i], none);
    const uint32_t keep = group_kept(t1, t2, ch.spread);
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (!(keep >> (group_of(e0 + j, ch.recip) << ch.spread & 31) & 1u)) key[j] = none;
    sk = s_keys[warp];          // the logits stay as they are
    __syncwarp();
    store_values(sk + e0, key);
    __syncwarp();               // expert() reads other lanes' keys
  }
  sort_descending(key);
  if (grouped && ch.own >= 0) {
    const uint32_t keep = group_kept(key[0], VPL > 1 ? key[VPL > 1 ? 1 : 0] : none, ch.own);
    if (!(keep >> (lane >> ch.own << ch.own) & 1u)) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = none;
    }
  }

  // The largest keys, slot i's key and lane in lane i; with a bias one more, to see
  // that the last one's lead is certain.  A lane's sorted keys wait in shared memory.
  const float* queue = s_queue[warp] + lane;
#pragma unroll
  for (int j = 1; j < VPL; ++j) s_queue[warp][32 * j + lane] = key[j];
  s_queue[warp][32 * VPL + lane] = none;
  float head = key[0], slot_key = none;
  int slot_lane = 0;
  auto pop = [&](int slot) {
    const float largest = redux_max(head);
    const int from = __ffs(__ballot_sync(FULL, head == largest)) - 1;
    if (lane == slot) {
      slot_key = largest;
      slot_lane = from;
    }
    if (lane == from && largest > none) {
      queue += 32;
      head = *queue;
    }
    return largest;
  };
  float past = none;
#pragma unroll 4
  for (int r = 0; r < a.slots; ++r) pop(r);
  if (a.bias) past = pop(a.slots);
  int found = a.slots + (a.bias ? 1 : 0);      // some of them may be -inf: no expert
  // The expert of a slot: the key's place among its lane's, and where the lane had
  // that key before, its next place.
  auto expert = [&]() {
    const float before = __shfl_up_sync(FULL, slot_key, 1);
    const int before_lane = __shfl_up_sync(FULL, slot_lane, 1);
    int skip = 0;
    if (__any_sync(FULL, lane > 0 && lane < found && slot_key > none && before == slot_key &&
                             before_lane == slot_lane))
      for (int i = 0; i < found && i < 32; ++i) {
        const float k = __shfl_sync(FULL, slot_key, i);
        const int from = __shfl_sync(FULL, slot_lane, i);
        skip += i < lane && k == slot_key && from == slot_lane;
      }
    int e = -1;
    if (lane < found && slot_key > none) {
      float k[VPL];
      load_values<VPL>(sk + slot_lane * VPL, true, k);
#pragma unroll
      for (int j = VPL - 1; j >= 0; --j)
        if (k[j] == slot_key) e = slot_lane * VPL + j;
      if (skip > 0) {
        e = -1;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
          if (k[j] == slot_key && e < 0 && skip-- == 0) e = slot_lane * VPL + j;
      }
    }
    return e;
  };
  int chosen = expert();
  if (a.bias && !unsure) {
    // Keys off by err and a rounding each.
    float q = __shfl_down_sync(FULL, slot_key, 1);
    if (lane == a.slots - 1) q = past;
    const float limit = 2.0f * err + 1.2e-7f * (fabsf(slot_key) + fabsf(q));
    const bool near = lane < a.slots && q > none && slot_key - q <= limit;
    if (__any_sync(FULL, near)) {
      // The same logit and bias are a true tie, in the order of the experts.
      const float x = chosen >= 0 ? sl[chosen] : none, b = chosen >= 0 ? a.bias[chosen] : 0.0f;
      const float x2 = __shfl_down_sync(FULL, x, 1), b2 = __shfl_down_sync(FULL, b, 1);
      bool differ = near && (lane == 31 || x != x2 || b != b2);
      // A tie of the last slot and the next key may hide others that are as near behind
      // it: any expert within the limit that is not tied with them.
      if (!__any_sync(FULL, differ) && __shfl_sync(FULL, near, a.slots - 1)) {
        const float last = __shfl_sync(FULL, slot_key, a.slots - 1);
        const float xl = __shfl_sync(FULL, x, a.slots - 1), bl = __shfl_sync(FULL, b, a.slots - 1);
#pragma unroll 1
        for (int e = lane; e < a.experts; e += 32) {
          const float k = sk[e];          // (larger ones are chosen, or of groups not kept)
          if (k > none && k <= last && last - k <= 2.0f * err + 1.2e-7f * (fabsf(last) + fabsf(k)))
            differ = differ || sl[e] != xl || a.bias[e] != bl;
        }
      }
      if (__any_sync(FULL, differ)) {
        const float last = __shfl_sync(FULL, slot_key, a.slots - 1);
        const float border = last - 2.0f * (2.0f * err + 2.4e-7f * fabsf(last));
        // Every expert that may be among the chosen, a lane each.
        float k = past;
        while (found < 32 && k >= border) k = pop(found++);
        if (k < border) {
          // Those below the border at the end, -inf among them, do no harm.
          chosen = expert();
          // A softmax's score is off by 2^-22 and 2.5 2^-24 |l - top| of itself, by what the
          // sum is (2^-22, the same of the mean |l - top| <= ln 512, 21 additions) and two
          // roundings: far less than err where it is small.  Whether each slot's key leads
          // those behind it by that is seen without 64 bits (8192 tokens, 8 of 256 with a
          // bias: 13.6 us, 14.6 without).
          const float l0 = chosen >= 0 ? sl[chosen] : none;
          // (From 88 on a score is 0 here, and the difference may be infinite.)
          const float apart = fminf(top - l0, 1000.0f);
          const float off = (sigmoid ? err : score(l0) * (3.0e-6f + 1.6e-7f * apart) + 2e-38f) +
                            2.4e-7f * fabsf(slot_key);
          float behind = __shfl_down_sync(FULL, chosen >= 0 ? slot_key + off : none, 1);
          if (lane == 31) behind = none;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const float o = __shfl_down_sync(FULL, behind, d);
            if (lane + d < 32) behind = fmaxf(behind, o);
          }
          if (__any_sync(FULL, lane < a.slots && chosen >= 0 && !(slot_key - off > behind)))
            chosen = choose_near(a, sl, top, chosen, __popc(__ballot_sync(FULL, chosen >= 0)));
        } else {
          unsure = true;
        }
      }
    }
  }
  if (unsure) chosen = choose_exactly<VPL>(ch, sl, top);
  if (lane >= a.slots) chosen = -1;

  // Weights.  Ratios are taken against the largest chosen score, so that no logit
  // is too small for them (the sums are between 1 / 2 and 512: quotients to 2 ulp).
  const bool real = chosen >= 0;
  const float li = real ? sl[chosen] : none;
  float w;
  if (sigmoid) {
    if (renorm) {
      const float low = real ? fminf(li, 0.0f) : none;
      const float best = redux_max(low);
      const float x = real ? sigmoid_n(li) * expf(low - best) : 0.0f;
      const float sum = warp_add(x);
      w = real ? __fdividef(x, sum) : 0.0f;
    } else {
      w = real ? sigmoid_of(li) : 0.0f;
    }
  } else if (renorm) {
    const float best = redux_max(li);
    const float x = real ? expf(li - best) : 0.0f;
    const float sum = warp_add(x);
    w = real ? __fdividef(x, sum) : 0.0f;
  } else {
    w = real ? __fdividef(expf(li - top), total) : 0.0f;
  }
  if (lane < a.slots) {
    ids[lane] = chosen;
    weights[lane] = w * a.scale;
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// With g = scale dweights: renormalised, w = s_i / sum s, c = sum_j g_j w_j and
//   softmax: dl_i = w_i (g_i - c),   sigmoid: dl_i = w_i (g_i - c) (1 - sigmoid(l_i));
// else sigmoid: dl_i = g_i s_i (1 - s_i),   softmax: dl_e = s_e (sum of g_i over the
// slots of e - sum_j g_j s_j), for every expert.
template <typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) moe_route_back_kernel(const RouteBackArgs a) {
  __shared__ float s_grad[ROUTE_WARPS][ROUTE_EXPERTS_MAX];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + warp;
  if (token >= a.tokens) return;
  const bool sigmoid = (a.flags & MXQ_ROUTE_SIGMOID) != 0;
  const bool renorm = (a.flags & MXQ_ROUTE_RENORM) != 0;
  const T* row = static_cast<const T*>(a.logits) + token * a.ldl;
  T* out = static_cast<T*>(a.dlogits) + token * a.ldd;
  float* sg = s_grad[warp];

  int e = -1;
  float g = 0.0f;
  if (lane < a.slots) {
    e = a.ids[token * a.slots + lane];
    if (e < 0 || e >= a.experts) e = -1;
    if (e >= 0) g = a.dweights[token * a.slots + lane] * a.scale;
  }
  const bool real = e >= 0;
  const float li = real ? load_logit(row + e) : -infinity();
  float d = 0.0f, share = 0.0f;     // the slot's part; softmax: sum_j g_j s_j
  if (!sigmoid && !renorm) {
    float top = -infinity(), total = 0.0f;
    for (int x = lane; x < a.experts; x += 32) {
      const float l = load_logit(row + x);
      sg[x] = l;
      top = fmaxf(top, l);
    }
    top = warp_max(top);
    if (!(top > -infinity())) top = 0.0f;
    for (int x = lane; x < a.experts; x += 32) {
      const float s = expf(sg[x] - top);
      sg[x] = s;
      total += s;
    }
    total = warp_add(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
    const float s = real ? expf(li - top) * inv : 0.0f;
    d = g * s;
    share = warp_add(d);
    // A token without an expert has no gradient, whatever its logits.
    for (int x = lane; x < a.experts; x += 32) sg[x] = share == 0.0f ? 0.0f : -(sg[x] * inv) * share;
  } else {
    for (int x = lane; x < a.experts; x += 32) sg[x] = 0.0f;
    if (!renorm) {
      d = real ? g * sigmoid_of(li) * sigmoid_of(-li) : 0.0f;
    } else {
      const float low = !real ? -infinity() : sigmoid ? fminf(li, 0.0f) : li;
      const float most = fmaxf(warp_max(low), -FLT_MAX);     // chosen scores may all be 0
      float x = real ? expf(low - most) : 0.0f;
      if (sigmoid && real) x *= sigmoid_n(li);
      const float sum = fmaxf(warp_add(x), 0.25f);           // 1 / 2 at least where one is not
      const float w = real ? x / sum : 0.0f;
      const float c = warp_add(g * w);
      d = w * (g - c);
      if (sigmoid && real) d *= sigmoid_of(-li);
    }
  }
  // An expert that has several slots gets the sum of their parts.
  float all = 0.0f;
  for (int j = 0; j < a.slots; ++j) {
    const int ej = __shfl_sync(FULL, e, j);
    const float dj = __shfl_sync(FULL, d, j);
    if (ej == e) all += dj;
  }
  __syncwarp();
  float base = real ? sg[e] : 0.0f;
  __syncwarp();
  if (real) sg[e] = base + all;     // slots of one expert write the same value
  __syncwarp();
  for (int x = lane; x < a.experts; x += 32) store_grad(out + x, sg[x]);
}

// ---------------------------------------------------------------------------
// Sorting
// ---------------------------------------------------------------------------

// A stable counting sort in one launch: the CTAs of one cluster take consecutive
// stretches of the pairs, and their warps consecutive parts of those.  A warp counts
// its pairs of each expert 32 at a time (lanes of the same expert find one another),
// which also gives each pair its rank; counts are summed over the warps and, through
// distributed shared memory, over the CTAs.  Pairs are then put in order in shared
// memory, so that `source` leaves in runs instead of 4 bytes a line.  131072 pairs over
// 256 experts 16 us (eight CTAs that read the pairs twice and scattered `source` 37 us),
// 32 pairs 4.8 us (device); past 262144 pairs, which registers do not hold, 524288 65 us and
// 2097152 243 us; what is left is shared memory's bank conflicts in 16 SMs,
// and a grid over all SMs would need a second launch and a workspace.
constexpr int SORT_CLUSTER = 16;
constexpr int SORT_ITEMS = 16;            // pairs a lane that are kept in registers
constexpr int64_t SORT_PER_CTA = 1024;    // pairs a CTA of 32 warps, as long as there are CTAs
constexpr int64_t SORT_SMALL = 1024;      // pairs that one CTA of 8 warps takes alone

// Counts [warps][E]; totals, sizes, first rows (E + 1), this CTA's first rows and first
// places, 32 words of a scan; a CTA's pairs in order, with their rows.
template <int WARPS>
struct SortShared {
  static constexpr int PAIRS = WARPS * 32 * SORT_ITEMS;
  __host__ __device__ static constexpr int words(int experts) {
    return ((WARPS + 5) * experts + 1 + 32 + 1) / 2 * 2;
  }
  __host__ __device__ static constexpr int bytes(int experts) { return 4 * words(experts) + 8 * PAIRS; }
};

// The cluster's barrier in two halves, for lanes that come apart: E experts and the rows
// past the last expert's end inside a warp, so that neither is the aligned form, which
// wants a whole warp at once.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) moe_sort_kernel(const SortArgs a) {
  constexpr int THREADS = 32 * WARPS;
  using L = SortShared<WARPS>;
  extern __shared__ __align__(16) int32_t smem[];
  const int E = a.experts;                  // at most THREADS
  int32_t* count = smem;                    // [warps][E]
  int32_t* total = count + WARPS * E;       // of this CTA, read by the others
  int32_t* sizes = total + E;               // of all
  int32_t* start = sizes + E;               // [E + 1] first rows
  int32_t* row0 = start + E + 1;            // this CTA's first rows
  int32_t* place0 = row0 + E;               // this CTA's first places in its own order
  int32_t* part = place0 + E;               // [32]
  int2* ordered = reinterpret_cast<int2*>(smem + L::words(E));
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), cta = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int64_t warps = static_cast<int64_t>(ctas) * WARPS;
  const int64_t seg = (a.n + 32 * warps - 1) / (32 * warps) * 32;
  const int64_t first = (static_cast<int64_t>(cta) * WARPS + warp) * seg;
  const int64_t last = first + seg < a.n ? first + seg : a.n;
  const bool held = seg <= 32 * SORT_ITEMS;
  int32_t* mine = count + warp * E;

  int32_t ids[SORT_ITEMS], rank[SORT_ITEMS];
  if (held) {
#pragma unroll
    for (int j = 0; j < SORT_ITEMS; ++j) {
      const int64_t i = first + 32 * j + lane;
      ids[j] = i < last ? a.ids[i] : -1;
    }
  }
  for (int i = tid; i < WARPS * E; i += THREADS) count[i] = 0;
  __syncthreads();
  auto real = [&](int e) { return e >= 0 && e < E ? e : -1; };
  // The place of the lane's pair among its warp's of expert e (-1: no pair).
  auto tally = [&](int e) {
    const uint32_t same = __match_any_sync(FULL, e);
    int32_t r = 0;
    if (e >= 0) r = mine[e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
    return r;
  };
  if (held) {
#pragma unroll
    for (int j = 0; j < SORT_ITEMS; ++j) {
      rank[j] = 0;
      if (first + 32 * j < last) {
        ids[j] = real(ids[j]);
        rank[j] = tally(ids[j]);
      }
    }
  } else {
    for (int64_t i = first; i < last; i += 32) tally(real(i + lane < last ? a.ids[i + lane] : -1));
  }
  __syncthreads();
  // Over the warps: a count becomes the sum of the earlier warps'.
  int32_t own = 0;
  if (tid < E) {
#pragma unroll 1
    for (int w0 = 0; w0 < WARPS; w0 += 8) {
      int32_t c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = count[(w0 + w) * E + tid];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        count[(w0 + w) * E + tid] = own;
        own += c[w];
      }
    }
    total[tid] = own;
  }
  cluster_arrive();
  cluster_wait();
  // Over the CTAs, and over the experts: first rows of padded groups, and first places.
  int32_t before = 0, size = 0;
  if (tid < E) {
#pragma unroll 4
    for (int r = 0; r < ctas; ++r) {
      const int32_t c = *cluster.map_shared_rank(total + tid, r);
      before += r < cta ? c : 0;
      size += c;
    }
  }
  // The other CTAs' totals have been read: they may leave once all have come here.
  cluster_arrive();
  const int32_t padded = (size + a.align - 1) / a.align * a.align;
  int32_t x = own, y = padded;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t ox = __shfl_up_sync(FULL, x, d), oy = __shfl_up_sync(FULL, y, d);
    if (lane >= d) {
      x += ox;
      y += oy;
    }
  }
  if (lane == 31 && warp < 16) {            // 512 experts at most
    part[warp] = x;
    part[16 + warp] = y;
  }
  __syncthreads();
  if (tid < E) {
    for (int w = 0; w < warp; ++w) {
      x += part[w];
      y += part[16 + w];
    }
    sizes[tid] = size;
    start[tid] = y - padded;
    row0[tid] = y - padded + before;
    place0[tid] = x - own;
    if (tid == E - 1) start[E] = y;
    if (cta == 0) {
      a.offsets[tid] = y - padded;
      if (tid == E - 1) a.offsets[E] = y;
      if (a.sizes) a.sizes[tid] = size;
    }
  }
  __syncthreads();
  if (held) {
#pragma unroll
    for (int j = 0; j < SORT_ITEMS; ++j) {
      const int64_t i = first + 32 * j + lane;
      if (i >= last) continue;
      const int e = ids[j];
      int32_t row = -1;
      if (e >= 0) {
        const int32_t r = mine[e] + rank[j];
        row = row0[e] + r;
        ordered[place0[e] + r] = make_int2(static_cast<int32_t>(i), row);
      }
      a.rows[i] = row;
    }
    if (a.source) {
      __syncthreads();
      const int pairs = place0[E - 1] + total[E - 1];
      for (int p = tid; p < pairs; p += THREADS) {
        const int2 v = ordered[p];
        a.source[v.y] = v.x;
      }
    }
  } else {
    for (int64_t i = first; i < last; i += 32) {
      const int e = real(i + lane < last ? a.ids[i + lane] : -1);
      const int32_t r = tally(e);
      const int32_t row = e >= 0 ? row0[e] + r : -1;
      if (i + lane < last) a.rows[i + lane] = row;
      if (e >= 0 && a.source) a.source[row] = static_cast<int32_t>(i + lane);
    }
  }
  if (a.source) {
    // Rows of no pair: those that pad an expert's, a warp an expert, and those past
    // the last expert's.
    for (int e = cta * WARPS + warp; e < E; e += static_cast<int>(warps))
      for (int32_t r = start[e] + sizes[e] + lane; r < start[e + 1]; r += 32) a.source[r] = -1;
    for (int64_t r = start[E] + static_cast<int64_t>(cta) * THREADS + tid; r < a.rows_max;
         r += static_cast<int64_t>(ctas) * THREADS)
      a.source[r] = -1;
  }
  cluster_wait();
}

template <int WARPS>
cudaError_t launch_sort_ctas(const SortArgs& a, unsigned ctas, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0}, wide{0};
  const void* kernel = reinterpret_cast<const void*>(moe_sort_kernel<WARPS>);
  cudaError_t e = allow_shared(kernel, SortShared<WARPS>::bytes(32 * WARPS < ROUTE_EXPERTS_MAX ? 32 * WARPS : ROUTE_EXPERTS_MAX), &allowed);
  if (e != cudaSuccess) return e;
  if (ctas > 8) {
    e = allow_clusters(kernel, &wide);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = SortShared<WARPS>::bytes(a.experts);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_sort_kernel<WARPS>, a);
}

// The largest n with 2^n <= x.
int log2_of(int x) {
  int n = 0;
  while (x > 1) {
    x >>= 1;
    ++n;
  }
  return n;
}

template <typename T, int VPL>
cudaError_t launch_route_v(Choice ch, cudaStream_t stream) {
  const RouteArgs& a = ch.a;
  auto wide = [](const void* p, int64_t row_bytes, int unit) {
    return reinterpret_cast<uintptr_t>(p) % unit == 0 && row_bytes % unit == 0;
  };
  ch.wide = wide(a.logits, a.ldl * sizeof(T), access_bytes<VPL, sizeof(T)>()) |
            wide(a.bias, 0, access_bytes<VPL, 4>()) << 1;
  // Groups that whole lanes hold, a power of two of them, are reduced by shuffles.
  const int lanes = ch.group_size / VPL;
  ch.own = ch.group_size % VPL == 0 && (lanes & (lanes - 1)) == 0 ? log2_of(lanes) : -1;
  const unsigned grid = static_cast<unsigned>((a.tokens + ROUTE_WARPS - 1) / ROUTE_WARPS);
  moe_route_kernel<T, VPL><<<grid, 32 * ROUTE_WARPS, 0, stream>>>(ch);
  return cudaGetLastError();
}

// As few experts a lane as hold them all: what a token costs grows with them (16384 tokens,
// 8 of 384 in groups 22 us with 12 and 36 with 16; 8 of 192 18.5 with 6 and 22.8 with 8).
template <typename T>
cudaError_t launch_route_t(const Choice& ch, cudaStream_t stream) {
  if (ch.a.experts <= 32) return launch_route_v<T, 1>(ch, stream);
  if (ch.a.experts <= 64) return launch_route_v<T, 2>(ch, stream);
  if (ch.a.experts <= 128) return launch_route_v<T, 4>(ch, stream);
  if (ch.a.experts <= 192) return launch_route_v<T, 6>(ch, stream);
  if (ch.a.experts <= 256) return launch_route_v<T, 8>(ch, stream);
  if (ch.a.experts <= 384) return launch_route_v<T, 12>(ch, stream);
  return launch_route_v<T, 16>(ch, stream);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  Choice ch{};
  ch.a = a;
  ch.group_size = a.experts / a.groups;
  ch.recip = ch.group_size == 1
                 ? 0u
                 : static_cast<uint32_t>((0x100000000ull + ch.group_size - 1) / ch.group_size);
  ch.spread = 5 - (a.groups == 1 ? 0 : log2_of(a.groups - 1) + 1);
  return (a.flags & MXQ_IN_F32) ? launch_route_t<float>(ch, stream)
                                : launch_route_t<uint16_t>(ch, stream);
}

cudaError_t launch_route_back(const RouteBackArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((a.tokens + ROUTE_WARPS - 1) / ROUTE_WARPS);
  if (a.flags & MXQ_IN_F32)
    moe_route_back_kernel<float><<<grid, 32 * ROUTE_WARPS, 0, stream>>>(a);
  else
    moe_route_back_kernel<uint16_t><<<grid, 32 * ROUTE_WARPS, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_sort(const SortArgs& a, cudaStream_t stream) {
  if (a.n <= SORT_SMALL && a.experts <= 256) return launch_sort_ctas<8>(a, 1, stream);
  const int64_t ctas = (a.n + SORT_PER_CTA - 1) / SORT_PER_CTA;
  return launch_sort_ctas<32>(a, ctas <= 1 ? 1 : ctas <= 2 ? 2 : ctas <= 4 ? 4 : ctas <= 8 ? 8 : SORT_CLUSTER, stream);
}

}  // namespace mxq
