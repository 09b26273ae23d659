// Group-limited routing with a balance bias, and the gradient of its weights.
//
// Per token, over the E_r units u with logit l_u (fp32):
//   s_u = 1 / (1 + exp(-l_u))            or  exp(l_u - max l) / sum exp(l - max l)
//   c_u = s_u + b_u                       b: balance bias, selection only
//   G_g = sum of the group_best (1 or 2) largest c of group g (consecutive units)
//   the groups_kept best groups stay; the k_t largest c inside them are selected
//   w_u = route_scale * s_u / (renorm ? sum of the selected s : 1)
// Ties go to the lower group and the lower unit.  A logit of -inf takes its
// unit out (NaN and +inf do too, and are reported).
//
// Gradient, with g_j the gradient of w_j (the selection is held fixed):
//   sigmoid          dl_j = route_scale g_j s_j (1 - s_j)
//   sigmoid, renorm  dl_j = route_scale w'_j (1 - s_j) (g_j - sum_i g_i w'_i)
//   softmax          dl_u = s_u (d_u - sum_i d_i s_i),  d_j = route_scale g_j, else 0
//   softmax, renorm  dl_j = route_scale w'_j (g_j - sum_i g_i w'_i)
// with w' = s / (sum of the selected s).  A softmax renormalised over the
// selection is the softmax of the selected logits alone, so that form needs
// neither the other logits nor their sum.  A renormalised sigmoid takes the
// common factor exp(m), m = min(max selected l, 0), out of every s.  Neither can
// divide by a sum that underflowed.
#include <cuda_fp16.h>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kWarps = 8;            // tokens of a CTA at a time
constexpr int kMaxWarps = 16;        // the same where that makes more CTAs than SMs
constexpr int kMaxUnits = 256;
constexpr int kMostGroups = kMaxUnits / 32;   // groups of a lane where it has several
constexpr unsigned kAll = 0xffffffffu;

// A token's list of units (score, unit).  Its space also holds the ranks of more
// than 32 groups, which are read by 16 bytes.
struct alignas(16) UnitList {
  float2 v[kMaxUnits];
};

__device__ __forceinline__ float warp_max_f32(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float warp_min_f32(float v) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}

// Sigmoids for the comparison, 1 / (1 + 2^(-l log2 e)) with the approximate
// exponential and reciprocal, each good to 2^-22 of its value: within 1e-6 of the
// value, 0 below 2^-126.  The rounding of l log2 e, which would add |l| 2^-24 and let
// neighbouring logits below -44 tie, is known exactly and goes into the sum by its
// first order, two units at a time (16384 tokens of 256 units 15.3 us; 15.2 without it, 16.3
// with expf).  |l| <= kLargeLogit.  The weights that leave the kernel are computed again with expf and a
// division.
__device__ __forceinline__ float2 sigmoids(float2 l) {
  constexpr float kHigh = 1.44269502f, kLow = 1.92596299e-8f;    // log2 e
  auto two = [](float v) { return make_float2(v, v); };
  const float2 t = __fmul2_rn(l, two(kHigh));
  const float2 rest = __ffma2_rn(l, two(-kLow), __ffma2_rn(l, two(-kHigh), t));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(-t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(-t.y));
  const float2 d = __ffma2_rn(e, __ffma2_rn(rest, two(0.693147181f), two(1.f)), two(1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return r;
}
constexpr float kLargeLogit = 1e38f;

// s(l) exp(-m) with m = min(largest selected l, 0), the same in every lane:
// l > 0 only where m = 0.
__device__ __forceinline__ float sigmoid_over(float l, float m) {
  const float e = expf(-fabsf(l));
  float top = l > 0.f ? 1.f : e;
  if (m < 0.f) top = expf(l - m);
  return top / (1.f + e);
}

struct GroupParams {
  const float* P;         // S partial logit arrays [S][T][E]
  int S;
  long long slice;        // T * E
  const float* bias;      // nullable: added to the logits of unit u, bias[u / n_sub]
  int n_sub;
  float* logits_out;      // nullable
  const int32_t* kpt;
  int T, E, k_max, score, renorm;
  float scale;
  int G, kept, best;
  const float* sel_bias;  // nullable
  int size;               // units per group
  int L;                  // lanes per group (MANY: 1)
  int gpl;                // groups per lane (1 unless MANY)
  int per;                // units per lane
  int vec;                // lanes hold aligned multiples of four units: 16-byte loads
  int32_t* idx;
  float* w;
  int32_t* k_out;         // nullable
  int32_t* load;          // nullable
  int zeroed;             // more than one CTA adds to load: a launch before this one clears it
  int32_t* status;
};

// One warp per token.  G <= 32: a group takes L = floor(32 / G) neighbouring
// lanes, each with `per` consecutive units, so units ascend with the lanes and
// a group's two best come from its lanes' two best.  MANY (G > 32): a lane
// holds whole groups, at most 16 units.
// Selection without a sort: k of the lanes' best units reach a bound, so the k
// best units do; the units that reach it, a few more than k, are listed and each
// counts the listed units before it.  The bound is found by counting in fp16,
// two lanes' heads at a time (k rounds of a warp maximum took 2 us more).
// Bound: issue slots and, before them, the chain through a token: 32 warps a SM
// keep both apart.  16384 tokens of 256 units in 8 groups, 4 kept, k = 8, with
// load counts: 15.6 us, 1.2 TB/s (sorting every lane and popping k heads: 24.7);
// one token 3.5 us, which is the launch and one chain.
template <int IPL, bool MANY>
__global__ void __launch_bounds__(kMaxWarps * 32) group_route_kernel(const GroupParams p) {
  __shared__ int32_t s_load[kMaxUnits];
  __shared__ UnitList s_list[kMaxWarps];
  __shared__ int32_t s_sel[kMaxWarps][32];
  __shared__ __align__(16) __half s_head[kMaxWarps][32];
  // With `zeroed` the kernel before this one clears `load`, after it has itself
  // waited for everything before: only `load` is waited for, at the end.
  if (!p.zeroed) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.load != nullptr) {
    for (int i = threadIdx.x; i < p.E; i += blockDim.x) s_load[i] = 0;
    __syncthreads();
  }
  // this lane's units [u0, u0 + n)
  const int g = MANY ? lane * p.gpl : lane / p.L;
  const int j = MANY ? 0 : lane - g * p.L;
  int u0 = g * p.size + j * p.per, n;
  if (MANY)
    n = max(0, min(p.per, p.E - u0));
  else
    n = g < p.G ? max(0, min(p.per, p.size - j * p.per)) : 0;
  if (n == 0) u0 = 0;
  // a NaN bias is reported and takes its unit out, as -inf does
  float b[IPL];
  bool bad_bias = false;
#pragma unroll
  for (int i = 0; i < IPL; ++i) {
    b[i] = i < n ? (p.sel_bias != nullptr ? __ldg(p.sel_bias + u0 + i) : 0.f) : -INFINITY;
    if (b[i] != b[i]) {
      bad_bias = true;
      b[i] = -INFINITY;
    }
  }
  if (bad_bias) report(p.status, MOE_ERR_NONFINITE);

  const int warps = blockDim.x >> 5;
  for (int t = blockIdx.x * warps + warp; t < p.T; t += gridDim.x * warps) {
    int k = p.kpt != nullptr ? __ldg(p.kpt + t) : p.k_max;
    const float* row = p.P + static_cast<size_t>(t) * p.E;
    float c[IPL];
    if (p.vec) {
#pragma unroll
      for (int i = 0; i < IPL; i += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) v = __ldg(reinterpret_cast<const float4*>(row + u0 + i));
        c[i] = v.x;
        if (i + 1 < IPL) c[i + 1] = v.y;
        if (i + 2 < IPL) c[i + 2] = v.z;
        if (i + 3 < IPL) c[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < IPL; ++i) c[i] = i < n ? __ldg(row + u0 + i) : 0.f;
    }
    for (int s = 1; s < p.S; ++s) {
#pragma unroll
      for (int i = 0; i < IPL; ++i)
        if (i < n) c[i] += __ldg(row + s * p.slice + u0 + i);
    }
    if (p.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < IPL; ++i)
        if (i < n) c[i] += __ldg(p.bias + (u0 + i) / p.n_sub);
    }
    if (p.logits_out != nullptr) {
      float* lo = p.logits_out + static_cast<size_t>(t) * p.E + u0;
#pragma unroll
      for (int i = 0; i < IPL; ++i)
        if (i < n) lo[i] = c[i];
    }
    if (k < 1 || k > p.k_max) {
      if (lane == 0) report(p.status, MOE_ERR_K_RANGE);
      k = min(max(k, 0), p.k_max);
    }
    // NaN and +inf are reported and leave the unit out, like -inf; a sigmoid's logits
    // past kLargeLogit, whose products overflow, count as that
    bool odd = false;
#pragma unroll
    for (int i = 0; i < IPL; ++i) odd |= !(fabsf(c[i]) < kLargeLogit);
    const bool masked = __any_sync(kAll, odd);
    unsigned out = 0u;               // bit i: unit i is out
    if (masked) {
      bool bad = false;
#pragma unroll
      for (int i = 0; i < IPL; ++i) {
        if (!(c[i] < INFINITY)) {
          bad = true;
          c[i] = -INFINITY;
        }
        if (c[i] == -INFINITY) out |= 1u << i;
        if (p.score != MOE_SCORE_SOFTMAX) c[i] = fminf(fmaxf(c[i], -kLargeLogit), kLargeLogit);
      }
      if (bad) report(p.status, MOE_ERR_NONFINITE);
    }
    // biased scores; the units past n are out by their b
    float mx = 0.f, sum = 1.f;
    if (p.score == MOE_SCORE_SOFTMAX) {
      mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < IPL; ++i)
        if (i < n) mx = fmaxf(mx, c[i]);
      mx = warp_max_f32(mx);
      const float m0 = mx > -INFINITY ? mx : 0.f;
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < IPL; ++i) {
        c[i] = i < n ? expf(c[i] - m0) : 0.f;
        part += c[i];
      }
      sum = warp_sum_f32(part);
      const float inv = sum > 0.f ? __fdividef(1.f, sum) : 1.f;
#pragma unroll
      for (int i = 0; i < IPL; ++i) c[i] = fmaf(c[i], inv, b[i]);
    } else {
#pragma unroll
      for (int i = 0; i < IPL; i += 2) {
        const float2 r = sigmoids(make_float2(c[i], i + 1 < IPL ? c[i + 1] : 0.f));
        c[i] = r.x + b[i];
        if (i + 1 < IPL) c[i + 1] = r.y + b[i + 1];
      }
    }
    if (masked) {
#pragma unroll
      for (int i = 0; i < IPL; ++i)
        if (out >> i & 1u) c[i] = -INFINITY;
    }

    if (MANY && p.kept < p.G) {
      float* rank = reinterpret_cast<float*>(s_list[warp].v);
      for (int q = 0; q < p.gpl; ++q) {
        float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < IPL; ++i)
          if (i < n && static_cast<unsigned>(i - q * p.size) < static_cast<unsigned>(p.size)) {
            a2 = fmaxf(a2, fminf(a1, c[i]));
            a1 = fmaxf(a1, c[i]);
          }
        if (g + q < p.G) rank[g + q] = a1 + (p.best == 2 && a2 > -INFINITY ? a2 : 0.f);
      }
      __syncwarp();
      // Groups ahead of each of the lane's: counted in fp16, two at a time.  Larger
      // as fp16 is larger, so the groups with fewer than `kept` such ahead are
      // the ones that stay and those that tie with the last of them; the ties, if
      // there are more than `kept`, are counted exactly.
      __half* coarse = reinterpret_cast<__half*>(rank + kMaxUnits);
      for (int o = lane; o < 256; o += 32) coarse[o] = __float2half_rn(o < p.G ? rank[o] : -INFINITY);
      __syncwarp();
      __half2 own[kMostGroups], ahead[kMostGroups];
#pragma unroll
      for (int q = 0; q < kMostGroups; ++q) {
        own[q] = __half2half2(coarse[min(g + q, 255)]);
        ahead[q] = __float2half2_rn(0.f);
      }
      for (int o = 0; o < p.G; o += 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(coarse + o);
#pragma unroll
        for (int q = 0; q < kMostGroups; ++q) {
          if (q >= p.gpl) break;
          ahead[q] = __hadd2(ahead[q], __hadd2(__hgt2(as_half2(v.x), own[q]), __hgt2(as_half2(v.y), own[q])));
          ahead[q] = __hadd2(ahead[q], __hadd2(__hgt2(as_half2(v.z), own[q]), __hgt2(as_half2(v.w), own[q])));
        }
      }
      int stay = 0;
      unsigned in = 0u;
#pragma unroll
      for (int q = 0; q < kMostGroups; ++q) {
        const bool mine = q < p.gpl && g + q < p.G &&
                          __low2float(ahead[q]) + __high2float(ahead[q]) < static_cast<float>(p.kept);
        stay += __popc(__ballot_sync(kAll, mine));
        if (mine) in |= 1u << q;
      }
      if (stay > p.kept) {
        for (int q = 0; q < p.gpl; ++q) {
          if (!(in >> q & 1u)) continue;
          const float mine = rank[g + q];
          int before = 0;
          for (int o = 0; o < p.G; ++o) before += rank[o] > mine || (rank[o] == mine && o < g + q);
          if (before >= p.kept) in &= ~(1u << q);
        }
      }
      for (int q = 0; q < p.gpl; ++q) {
        if (in >> q & 1u) continue;
#pragma unroll
        for (int i = 0; i < IPL; ++i)
          if (static_cast<unsigned>(i - q * p.size) < static_cast<unsigned>(p.size)) c[i] = -INFINITY;
      }
      __syncwarp();
    }
    // the lane's two best
    float a1 = c[0], a2 = -INFINITY;
#pragma unroll
    for (int i = 1; i < IPL; ++i) {
      a2 = fmaxf(a2, fminf(a1, c[i]));
      a1 = fmaxf(a1, c[i]);
    }
    float head = a1;
    if (!MANY && p.kept < p.G) {
      if ((p.L & (p.L - 1)) == 0) {
        for (int off = 1; off < p.L; off <<= 1) {
          const float b1 = __shfl_xor_sync(kAll, a1, off), b2 = __shfl_xor_sync(kAll, a2, off);
          a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
          a1 = fmaxf(a1, b1);
        }
      } else {
        const float h1 = a1, h2 = a2;
        a1 = a2 = -INFINITY;
        for (int o = 0; o < p.L; ++o) {
          const int from = min(g * p.L + o, 31);
          const float b1 = __shfl_sync(kAll, h1, from), b2 = __shfl_sync(kAll, h2, from);
          a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
          a1 = fmaxf(a1, b1);
        }
      }
      const float rank = a1 + (p.best == 2 && a2 > -INFINITY ? a2 : 0.f);
      int ahead = 0;
#pragma unroll 8
      for (int o = 0; o < p.G; ++o) {
        const float other = __shfl_sync(kAll, rank, o * p.L);
        ahead += other > rank || (other == rank && o < g);
      }
      if (ahead >= p.kept) {
        head = -INFINITY;
#pragma unroll
        for (int i = 0; i < IPL; ++i) c[i] = -INFINITY;
      }
    }
    // the bound: the least head of the lanes with fewer than k larger ones, where
    // larger is larger as fp16 (never more lanes than the k best leave out)
    __half* heads = s_head[warp];
    heads[lane] = __float2half_rn(head);
    __syncwarp();
    const __half2 own = __half2half2(heads[lane]);
    __half2 larger = __float2half2_rn(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(heads)[i];
      larger = __hadd2(larger, __hgt2(as_half2(v.x), own));
      larger = __hadd2(larger, __hgt2(as_half2(v.y), own));
      larger = __hadd2(larger, __hgt2(as_half2(v.z), own));
      larger = __hadd2(larger, __hgt2(as_half2(v.w), own));
    }
    const float before = __low2float(larger) + __high2float(larger);
    const float bound = warp_min_f32(before < static_cast<float>(k) ? head : INFINITY);
    // the units that reach it, in any order
    const float least = bound > -INFINITY ? bound : -3.402823466e38f;
    int listed = 0;
#pragma unroll
    for (int i = 0; i < IPL; ++i) listed += c[i] >= least;
    int to = listed;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kAll, to, off);
      if (lane >= off) to += o;
    }
    const int mine_n = listed;
    listed = __shfl_sync(kAll, to, 31);
    to -= mine_n;
#pragma unroll
    for (int i = 0; i < IPL; ++i)
      if (c[i] >= least) s_list[warp].v[to++] = make_float2(c[i], __int_as_float(u0 + i));
    __syncwarp();
    const int got = min(k, listed);
    for (int i = lane; i < listed; i += 32) {
      const float2 mine = s_list[warp].v[i];
      const int unit = __float_as_int(mine.y);
      int ahead = 0;
#pragma unroll 4
      for (int o = 0; o < listed; ++o) {
        const float2 other = s_list[warp].v[o];
        ahead += other.x > mine.x || (other.x == mine.x && __float_as_int(other.y) < unit);
      }
      if (ahead < got) s_sel[warp][ahead] = unit;
    }
    __syncwarp();
    // weights of the selected units, one per lane, from their logits
    const bool sel = lane < got;
    const int unit = sel ? s_sel[warp][lane] : -1;
    float l = -INFINITY;
    if (sel) {
      l = __ldg(row + unit);
      for (int s = 1; s < p.S; ++s) l += __ldg(row + s * p.slice + unit);
      if (p.bias != nullptr) l += __ldg(p.bias + unit / p.n_sub);
    }
    float wt = 0.f;
    if (p.score == MOE_SCORE_SOFTMAX) {
      const float top = p.renorm ? warp_max_f32(l) : mx;
      const float e = sel ? expf(l - top) : 0.f;
      const float total = p.renorm ? warp_sum_f32(e) : sum;
      if (sel) wt = e / total;
    } else {
      const float m = p.renorm ? fminf(warp_max_f32(l), 0.f) : 0.f;
      const float s = sel ? sigmoid_over(l, m) : 0.f;
      const float total = p.renorm ? warp_sum_f32(s) : 1.f;
      if (sel) wt = s / total;
    }
    if (lane < p.k_max) {
      const size_t o = static_cast<size_t>(t) * p.k_max + lane;
      p.idx[o] = unit;
      p.w[o] = wt * p.scale;
    }
    if (p.k_out != nullptr && lane == 0) p.k_out[t] = got;
    if (p.load != nullptr && sel) atomicAdd(&s_load[unit], 1);
    __syncwarp();   // the lists are written again for the next token
  }
  if (p.load != nullptr) {
    __syncthreads();
    if (p.zeroed) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = threadIdx.x; i < p.E; i += blockDim.x) {
      const int v = s_load[i];
      if (gridDim.x == 1)
        p.load[i] = v;
      else if (v != 0)
        atomicAdd(p.load + i, v);
    }
  }
}

__global__ void __launch_bounds__(kMaxUnits) zero_load_kernel(int32_t* load, int E) {
  pdl_wait_and_trigger();
  if (static_cast<int>(threadIdx.x) < E) load[threadIdx.x] = 0;
}

struct RouteBackParams {
  const float* logits;
  const int32_t* idx;
  const float* d_w;
  float* d_logits;
  int T, E, k_max, score, renorm;
  float scale;
  int vec;                // E % 4 == 0 and 16-byte aligned rows
  int32_t* status;
};

// One warp per token: lane j takes slot j.  The softmax that is not renormalised
// has a row of gradients: its logits are in registers, NV a lane, read once.
// The others (NV = 0) have k: their row leaves through shared memory, whole.
// Bound: latency, of which occupancy hides most (40 registers for the others: 5.2
// us, 48: 6.1).  16384 tokens of 128 units, k = 8: 4.9 us dense (3.6 TB/s; with a
// row in eight registers a lane whatever its length 7.0), 5.1 renormalised.
template <int NV>
__global__ void __launch_bounds__(kWarps * 32, NV == 0 ? 6 : 4) route_backward_kernel(const RouteBackParams p) {
  __shared__ __align__(16) float s_row[kWarps][kMaxUnits];
  pdl_wait_and_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* d = s_row[warp];
  for (int t = blockIdx.x * kWarps + warp; t < p.T; t += gridDim.x * kWarps) {
    const float* row = p.logits + static_cast<size_t>(t) * p.E;
    float* out = p.d_logits + static_cast<size_t>(t) * p.E;
    int u = -1;
    float gw = 0.f;
    if (lane < p.k_max) {
      const size_t o = static_cast<size_t>(t) * p.k_max + lane;
      u = p.idx[o];
      gw = p.d_w[o];
    }
    float v[NV + 1];
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        v[j] = lane + 32 * j < p.E ? __ldg(row + lane + 32 * j) : -INFINITY;
    }
    for (int i = lane; i < p.E; i += 32) d[i] = 0.f;
    __syncwarp();
    // a unit listed twice has two slots for its mark
    int* mark = reinterpret_cast<int*>(d);
    bool wrong = u >= p.E || u < -1;
    if (wrong) u = -1;
    if (u >= 0) mark[u] = lane;
    __syncwarp();
    if (u >= 0 && mark[u] != lane) wrong = true;
    if (__any_sync(kAll, wrong)) {
      if (wrong) report(p.status, MOE_ERR_BAD_INDEX);
      if ((__match_any_sync(kAll, u) & ((1u << lane) - 1u)) != 0u) u = -1;   // the first slot stays
    }
    __syncwarp();
    bool bad = false;
    if constexpr (NV > 0) {
      if (u >= 0) d[u] = gw * p.scale;
      float mx = -INFINITY, sum = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!(v[j] < INFINITY)) {
          bad = true;
          v[j] = -INFINITY;
        }
        mx = fmaxf(mx, v[j]);
      }
      mx = warp_max_f32(mx);
      __syncwarp();
      if (!(mx > -INFINITY)) mx = 0.f;
      float dv[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        // a unit that is out has no part, whatever a slot says
        dv[j] = v[j] > -INFINITY ? d[lane + 32 * j] : 0.f;
        v[j] = expf(v[j] - mx);
        sum += v[j];
        dot += v[j] * dv[j];
      }
      sum = warp_sum_f32(sum);
      dot = warp_sum_f32(dot);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      dot *= inv;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (lane + 32 * j < p.E) out[lane + 32 * j] = v[j] * inv * (dv[j] - dot);
    } else {
      float l = u >= 0 ? __ldg(row + u) : -INFINITY;
      bad = !(l < INFINITY);
      if (bad) l = -INFINITY;
      const bool sel = u >= 0 && l > -INFINITY;
      if (!sel) gw = 0.f;
      float dl;
      if (p.score == MOE_SCORE_SOFTMAX) {
        const float top = warp_max_f32(l);
        const float e = sel ? expf(l - top) : 0.f;
        const float total = warp_sum_f32(e);
        const float wt = sel ? e / total : 0.f;
        const float dot = warp_sum_f32(gw * wt);
        dl = p.scale * wt * (gw - dot);
      } else {
        const float m = p.renorm ? fminf(warp_max_f32(l), 0.f) : 0.f;
        const float s = sel ? sigmoid_over(l, m) : 0.f;
        const float ms = 1.f / (1.f + expf(l));        // 1 - s without cancellation
        float wt = s, dot = 0.f;
        if (p.renorm) {
          const float total = warp_sum_f32(s);
          if (sel) wt = s / total;
          dot = warp_sum_f32(gw * wt);
        }
        dl = p.scale * wt * ms * (gw - dot);
      }
      if (u >= 0) d[u] = sel ? dl : 0.f;
      __syncwarp();
      if (p.vec) {
        for (int i = lane; i < p.E / 4; i += 32)
          reinterpret_cast<float4*>(out)[i] = reinterpret_cast<const float4*>(d)[i];
      } else {
        for (int i = lane; i < p.E; i += 32) out[i] = d[i];
      }
    }
    if (bad) report(p.status, MOE_ERR_NONFINITE);
    __syncwarp();
  }
}

inline bool aligned16p(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

}  // namespace

cudaError_t launch_group_route(const GroupRouteArgs& a, cudaStream_t s) {
  if (a.T == 0) {
    if (a.load != nullptr) return cudaMemsetAsync(a.load, 0, sizeof(int32_t) * a.E_r, s);
    return cudaSuccess;
  }
  GroupParams p{};
  p.P = a.partial;
  p.S = a.S;
  p.slice = static_cast<long long>(a.T) * a.E_r;
  p.bias = a.bias;
  p.n_sub = a.n_sub;
  p.logits_out = a.logits_out;
  p.kpt = a.k_per_token;
  p.T = a.T;
  p.E = a.E_r;
  p.k_max = a.k_max;
  p.score = a.score;
  p.renorm = a.renorm;
  p.scale = a.route_scale;
  p.G = a.n_groups;
  p.kept = a.groups_kept;
  p.best = a.group_best;
  // with every group kept the grouping decides nothing
  if (p.kept == p.G) p.G = p.kept = 1;
  p.sel_bias = a.select_bias;
  p.size = p.E / p.G;
  const bool many = p.G > 32;
  p.L = many ? 1 : 32 / p.G;
  p.gpl = many ? (p.G + 31) / 32 : 1;
  p.per = many ? p.gpl * p.size : (p.size + p.L - 1) / p.L;
  p.vec = p.per % 4 == 0 && p.size % 4 == 0 && aligned16p(a.partial);
  p.idx = a.topk_idx;
  p.w = a.topk_w;
  p.k_out = a.k_out;
  p.load = a.load;
  p.status = a.status;
  // 16 warps where there are more tokens than eight a SM: half as many CTAs add
  // to the same load counts (256 units, with 8 and 16: 600 tokens 4.5, 4.9 us;
  // 2400 5.4, 5.2; 4096 8.5, 7.1; 16384 17.7, 15.8).  32 warps a SM: 16384 tokens
  // take 15.9 us, 19.6 with 16 and 20.2 with 48.
  const int warps = a.T > kWarps * a.sm_count ? kMaxWarps : kWarps;
  const int blocks = (a.T + warps - 1) / warps, most = 4 * kWarps / warps * a.sm_count;
  const int grid = blocks < most ? blocks : most;
  p.zeroed = a.load != nullptr && grid > 1;
  if (p.zeroed) {
    const cudaError_t e = launch_pdl(zero_load_kernel, dim3(1), dim3(kMaxUnits), 0, s, a.load, a.E_r);
    if (e != cudaSuccess) return e;
  }
  const dim3 g(grid), b(warps * 32);
  if (many) return launch_pdl(group_route_kernel<16, true>, g, b, 0, s, p);
  if (p.per <= 1) return launch_pdl(group_route_kernel<1, false>, g, b, 0, s, p);
  if (p.per <= 2) return launch_pdl(group_route_kernel<2, false>, g, b, 0, s, p);
  if (p.per <= 4) return launch_pdl(group_route_kernel<4, false>, g, b, 0, s, p);
  if (p.per <= 8) return launch_pdl(group_route_kernel<8, false>, g, b, 0, s, p);
  return launch_pdl(group_route_kernel<16, false>, g, b, 0, s, p);
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  RouteBackParams p{};
  p.logits = a.logits;
  p.idx = a.topk_idx;
  p.d_w = a.d_topk_w;
  p.d_logits = a.d_logits;
  p.T = a.T;
  p.E = a.E_r;
  p.k_max = a.k_max;
  p.score = a.score;
  p.renorm = a.renorm;
  p.scale = a.route_scale;
  p.vec = a.E_r % 4 == 0 && aligned16p(a.logits) && aligned16p(a.d_logits);
  p.status = a.status;
  const int blocks = (a.T + kWarps - 1) / kWarps;
  const int grid = blocks < 8 * a.sm_count ? blocks : 8 * a.sm_count;
  const dim3 g(grid), b(kWarps * 32);
  if (a.score != MOE_SCORE_SOFTMAX || a.renorm) return launch_pdl(route_backward_kernel<0>, g, b, 0, s, p);
  if (a.E_r <= 128) return launch_pdl(route_backward_kernel<4>, g, b, 0, s, p);
  return launch_pdl(route_backward_kernel<kMaxUnits / 32>, g, b, 0, s, p);
}

}  // namespace moe
