// The norms around a residual block, with its gate and scales, in one pass, and
// their gradients.
//
//   z  = y * rstd(y) * w_post            (z = y without a post-norm)
//   r' = rs * r + bs * g * z             rs, bs: residual and branch scale, g: gate
//   h  = r' * rstd(r') * w_pre           the next block's pre-norm
//   rstd(v) = 1 / sqrt(mean(v^2) + eps); every w has weight_offset added
//
// Gradients, D the whole gradient at r' (a = mean over the row):
//   D    = dr' + rstd (dh w_pre - m a(dh w_pre m)),          m = r' rstd(r')
//   dr   = rs D;   dz = bs g D;   dg = bs D z (summed over what g is shared by)
//   dy   = rstd(y) (dz w_post - n a(dz w_post n)),           n = y rstd(y)
//   dw_post = sum_t dz n;   dw_pre = sum_t dh m
// r' and both rstd are computed again from r, y and g: the row is in shared
// memory anyway, so the backward pass reads nothing that the forward pass
// would have had to store.  The sums of both norms' gradients are taken in one
// round, which rearranges a(dz w_post n) into three sums over r'.
//
// Bound: memory.  A group of TPR threads owns a row, EPT elements a thread, and
// walks over rows with a ring of row slots that bulk copies fill ahead.  Row
// sums cost a barrier each, so there is one round of them per row: sum(y^2) of
// the next row is taken with the sums of this one.  Rows of any alignment are
// copied as the 16-byte granules around them.
// Sums and everything between load and store are fp32; each output is rounded
// once.
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr uint32_t kSmemBudget = 200 * 1024;

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// A thread's EPT elements of a row of H.  VEC = 8: vectors of eight columns,
// (tid + v TPR) 8 ...; VEC = 1: columns tid + e TPR.
template <int VEC>
struct Cols {
  int tid, tpr, H;
  __device__ __forceinline__ int col(int e) const {
    return VEC == 1 ? tid + e * tpr : (tid + (e / VEC) * tpr) * VEC + e % VEC;
  }
};

// Elements past H come back 0 and are not stored.
template <typename T, int VEC, int EPT>
__device__ __forceinline__ void load_row(const T* __restrict__ p, const Cols<VEC>& c,
                                         float (&v)[EPT]) {
  if constexpr (VEC == 1) {
#pragma unroll
    for (int e = 0; e < EPT; ++e) v[e] = c.col(e) < c.H ? to_f<T>(p[c.col(e)]) : 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < EPT; e += 8) {
      const int at = c.col(e);
      if (at < c.H) {
        if constexpr (sizeof(T) == 2) {
          const uint4 q = *reinterpret_cast<const uint4*>(p + at);
          v[e] = bf16lo(q.x); v[e + 1] = bf16hi(q.x);
          v[e + 2] = bf16lo(q.y); v[e + 3] = bf16hi(q.y);
          v[e + 4] = bf16lo(q.z); v[e + 5] = bf16hi(q.z);
          v[e + 6] = bf16lo(q.w); v[e + 7] = bf16hi(q.w);
        } else {
          const float4 a = *reinterpret_cast<const float4*>(p + at);
          const float4 b = *reinterpret_cast<const float4*>(p + at + 4);
          v[e] = a.x; v[e + 1] = a.y; v[e + 2] = a.z; v[e + 3] = a.w;
          v[e + 4] = b.x; v[e + 5] = b.y; v[e + 6] = b.z; v[e + 7] = b.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[e + i] = 0.f;
      }
    }
  }
}

template <typename T, int VEC, int EPT>
__device__ __forceinline__ void store_row(T* __restrict__ p, const Cols<VEC>& c,
                                          const float (&v)[EPT]) {
  if constexpr (VEC == 1) {
#pragma unroll
    for (int e = 0; e < EPT; ++e)
      if (c.col(e) < c.H) p[c.col(e)] = from_f<T>(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < EPT; e += 8) {
      const int at = c.col(e);
      if (at < c.H) {
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<uint4*>(p + at) =
              make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]),
                         pack_bf16x2(v[e + 4], v[e + 5]), pack_bf16x2(v[e + 6], v[e + 7]));
        } else {
          *reinterpret_cast<float4*>(p + at) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          *reinterpret_cast<float4*>(p + at + 4) =
              make_float4(v[e + 4], v[e + 5], v[e + 6], v[e + 7]);
        }
      }
    }
  }
}

// A thread's elements of a row as they are in memory (bf16 two to a register),
// for what is kept across rows or sums.
template <typename T, int VEC, int EPT>
struct Kept;
template <int VEC, int EPT>
struct Kept<float, VEC, EPT> {
  float v[EPT];
  __device__ __forceinline__ void load(const float* p, const Cols<VEC>& c) {
    load_row<float, VEC, EPT>(p, c, v);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < EPT; ++e) v[e] = 0.f;
  }
  __device__ __forceinline__ float operator[](int e) const { return v[e]; }
};
template <int VEC, int EPT>
struct Kept<__nv_bfloat16, VEC, EPT> {
  uint32_t v[EPT / 2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const Cols<VEC>& c) {
    if constexpr (VEC == 1) {
      const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
      for (int e = 0; e < EPT; e += 2)
        v[e / 2] = (c.col(e) < c.H ? u[c.col(e)] : 0u) |
                   (c.col(e + 1) < c.H ? static_cast<uint32_t>(u[c.col(e + 1)]) << 16 : 0u);
    } else {
#pragma unroll
      for (int e = 0; e < EPT; e += 8) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (c.col(e) < c.H) q = *reinterpret_cast<const uint4*>(p + c.col(e));
        v[e / 2] = q.x;
        v[e / 2 + 1] = q.y;
        v[e / 2 + 2] = q.z;
        v[e / 2 + 3] = q.w;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < EPT / 2; ++e) v[e] = 0u;
  }
  __device__ __forceinline__ float operator[](int e) const {
    return (e & 1) ? bf16hi(v[e / 2]) : bf16lo(v[e / 2]);
  }
};

struct NormParams {
  int T, H;
  int tpr, groups, slots;       // threads per row, row groups per CTA, ring slots per group
  uint32_t pitch_r, pitch_a;    // bytes of a residual / activation row in a slot
  uint32_t slot_bytes;
  int gate;                     // moe_gate_kind
  float eps, offset, rs, bs;
  const void* r;
  const void* y;
  const void* gate_p;
  const void* w_post;
  const void* w_pre;
  long long ld_r, ld_y, ld_g, ld_out, ld_h;
  void* out;                    // r' (forward), dr (backward)
  void* h;                      // h (forward), dy (backward)
  // backward
  const void* d_out;
  const void* d_h;
  long long ld_dout, ld_dh;
  void* d_gate;
  float* part;                  // [grid][n_part][H]
  int n_part;
  int32_t* status;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The 16-byte granules around the `bytes` at p.
__device__ __forceinline__ uint32_t granules(const void* p, uint32_t bytes, const void** from) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), lo = a & ~static_cast<uintptr_t>(15);
  *from = reinterpret_cast<const void*>(lo);
  return static_cast<uint32_t>(((a + bytes + 15) & ~static_cast<uintptr_t>(15)) - lo);
}
__device__ __forceinline__ uint32_t skew(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
}

constexpr int kSumFloats = 8 * 32;    // up to eight sums of up to 32 warps

// Sums N (2 or 8) values over the group's threads, in a fixed order; every
// thread gets the sums.  `red` holds one buffer per parity: a buffer is written
// again only two sums later, behind the barrier of the sum between, which
// follows everyone's reads.
// Eight values fold into one per lane quad while they are added (9 shuffles
// instead of 40).
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int tpr, int bar, int tid, float* red,
                                          int& parity) {
  static_assert(N == 2 || N == 8, "two or eight sums");
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = tid & 31;
  // lane holds the sum of value lane * N / 32 over its warp
  float part;
  if constexpr (N == 8) {
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float keep = (lane & 16) ? v[i + 4] : v[i], send = (lane & 16) ? v[i] : v[i + 4];
      a[i] = keep + __shfl_xor_sync(kAll, send, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float keep = (lane & 8) ? a[i + 2] : a[i], send = (lane & 8) ? a[i] : a[i + 2];
      b[i] = keep + __shfl_xor_sync(kAll, send, 8);
    }
    const float keep = (lane & 4) ? b[1] : b[0], send = (lane & 4) ? b[0] : b[1];
    part = keep + __shfl_xor_sync(kAll, send, 4);
  } else {
    const float keep = (lane & 16) ? v[1] : v[0], send = (lane & 16) ? v[0] : v[1];
    part = keep + __shfl_xor_sync(kAll, send, 16);
    part += __shfl_xor_sync(kAll, part, 8);
    part += __shfl_xor_sync(kAll, part, 4);
  }
  part += __shfl_xor_sync(kAll, part, 2);
  part += __shfl_xor_sync(kAll, part, 1);
  if (tpr > 32) {
    constexpr int kLanes = 32 / N;      // lanes of a value
    float* buf = red + parity * kSumFloats;
    parity ^= 1;
    const int warp = tid >> 5, nw = tpr >> 5, value = lane / kLanes;
    if (lane % kLanes == 0) buf[value * 32 + warp] = part;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
    part = 0.f;
#pragma unroll
    for (int w = 0; w < 32; w += kLanes)
      if (w + lane % kLanes < nw) part += buf[value * 32 + w + lane % kLanes];
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) part += __shfl_xor_sync(kAll, part, off);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(kAll, part, i * (32 / N));
}

// Shared memory: [groups][slots] row slots, then the sum buffers, then barriers.
struct NormSmem {
  uint32_t red, bars, total;
};
__host__ __device__ inline NormSmem norm_smem(uint32_t slot_bytes, int slots, int groups) {
  NormSmem o;
  uint32_t b = slot_bytes * static_cast<uint32_t>(slots) * static_cast<uint32_t>(groups);
  o.red = b;
  b += static_cast<uint32_t>(groups) * 2 * kSumFloats * 4;
  o.bars = b;
  b += static_cast<uint32_t>(groups * slots) * 8;
  o.total = b;
  return o;
}

// One group's view of the ring: its rows are first, first + step, ...
template <typename R, typename A, bool BACK>
struct Ring {
  uint8_t* base;
  uint64_t* full;
  const NormParams* p;
  uint32_t bytes_r, bytes_a;

  __device__ __forceinline__ void fill_one(uint32_t at, const void* src, uint32_t bytes,
                                           uint64_t* bar, uint32_t& total, bool issue) const {
    const void* from;
    const uint32_t n = granules(src, bytes, &from);
    total += n;
    if (issue) bulk_load(at, from, n, bar);
  }
  __device__ __forceinline__ const R* r_row(int t) const {
    return static_cast<const R*>(p->r) + static_cast<long long>(t) * p->ld_r;
  }
  __device__ __forceinline__ const A* y_row(int t) const {
    return static_cast<const A*>(p->y) + static_cast<long long>(t) * p->ld_y;
  }
  __device__ __forceinline__ const A* g_row(int t) const {
    return static_cast<const A*>(p->gate_p) + static_cast<long long>(t) * p->ld_g;
  }
  __device__ __forceinline__ const R* dout_row(int t) const {
    return static_cast<const R*>(p->d_out) + static_cast<long long>(t) * p->ld_dout;
  }
  __device__ __forceinline__ const A* dh_row(int t) const {
    return static_cast<const A*>(p->d_h) + static_cast<long long>(t) * p->ld_dh;
  }
  // offsets of the rows inside a slot: r, y, [gate], [d_out], [d_h]
  __device__ __forceinline__ void fill(int slot, int t) const {
    uint64_t* bar = full + slot;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      uint32_t at = smem_u32(base) + static_cast<uint32_t>(slot) * p->slot_bytes, total = 0;
      const bool go = pass == 1;
      fill_one(at, r_row(t), bytes_r, bar, total, go);
      at += p->pitch_r;
      if (p->y != nullptr) fill_one(at, y_row(t), bytes_a, bar, total, go);
      at += p->pitch_a;
      if (p->gate == MOE_GATE_FULL) {
        fill_one(at, g_row(t), bytes_a, bar, total, go);
        at += p->pitch_a;
      }
      if (BACK) {
        if (p->d_out != nullptr) fill_one(at, dout_row(t), bytes_r, bar, total, go);
        at += p->pitch_r;
        if (p->d_h != nullptr) fill_one(at, dh_row(t), bytes_a, bar, total, go);
      }
      if (!go) mbar_expect_tx(bar, total);
    }
  }
};

template <typename R, typename A, int VEC, int EPT, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) block_norm_kernel(const NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const NormSmem L = norm_smem(p.slot_bytes, p.slots, p.groups);
  const int group = threadIdx.x / p.tpr, tid = threadIdx.x - group * p.tpr;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  float* red = reinterpret_cast<float*>(smem + L.red) + group * 2 * kSumFloats;
  Ring<R, A, false> ring;
  ring.base = smem + static_cast<uint32_t>(group * p.slots) * p.slot_bytes;
  ring.full = bars + group * p.slots;
  ring.p = &p;
  ring.bytes_r = static_cast<uint32_t>(p.H * sizeof(R));
  ring.bytes_a = static_cast<uint32_t>(p.H * sizeof(A));
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.groups * p.slots; ++i) mbar_init(bars + i, 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait_and_trigger();
  const int step = gridDim.x * p.groups;
  const int first = blockIdx.x + gridDim.x * group;
  if (tid == 0)
    for (int s = 0; s < p.slots; ++s)
      if (first + s * step < p.T) ring.fill(s, first + s * step);
  const Cols<VEC> c{tid, p.tpr, p.H};
  const bool post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  Kept<A, VEC, EPT> w_post, w_pre;
  w_post.zero();
  w_pre.zero();
  if (post) w_post.load(static_cast<const A*>(p.w_post), c);
  if (pre) w_pre.load(static_cast<const A*>(p.w_pre), c);
  const float inv_h = 1.f / static_cast<float>(p.H);
  const bool ahead = p.slots > 1;     // the next row is there while this one is at work
  int slot = 0, parity = 0;
  uint32_t phase = 0;
  Kept<A, VEC, EPT> x;                // y of the row
  float sq = 0.f;                     // its sum of squares
  auto take_y = [&](int t, int sl, uint32_t ph) {
    if (!mbar_wait(ring.full + sl, ph, nullptr)) report(p.status, MOE_ERR_DEVICE_TIMEOUT);
    const uint8_t* at = ring.base + static_cast<uint32_t>(sl) * p.slot_bytes + p.pitch_r;
    x.zero();
    if (p.y != nullptr) x.load(reinterpret_cast<const A*>(at + (VEC == 1 ? skew(ring.y_row(t)) : 0)), c);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) q += x[e] * x[e];
    return q;
  };
  for (int t = first; t < p.T; t += step) {
    if (t == first || !ahead) {
      float q[2] = {take_y(t, slot, phase), 0.f};
      group_sum<2>(q, p.tpr, 1 + group, tid, red, parity);
      sq = q[0];
    }
    float scale = p.bs;
    if (p.gate == MOE_GATE_TOKEN) scale *= to_f<A>(static_cast<const A*>(p.gate_p)[t]);
    if (post) scale *= rsqrtf(sq * inv_h + p.eps);
    const uint8_t* at = ring.base + static_cast<uint32_t>(slot) * p.slot_bytes;
    float v[EPT];
    load_row<R, VEC, EPT>(reinterpret_cast<const R*>(at + (VEC == 1 ? skew(ring.r_row(t)) : 0)), c, v);
    at += p.pitch_r + p.pitch_a;
    const A* gate = nullptr;
    if (p.gate == MOE_GATE_FULL)
      gate = reinterpret_cast<const A*>(at + (VEC == 1 ? skew(ring.g_row(t)) : 0));
    else if (p.gate == MOE_GATE_CHANNEL)
      gate = static_cast<const A*>(p.gate_p);
#pragma unroll
    for (int e = 0; e < EPT; ++e) v[e] *= p.rs;
    if (gate != nullptr) {
      Kept<A, VEC, EPT> g;
      g.load(gate, c);
#pragma unroll
      for (int e = 0; e < EPT; ++e) v[e] += x[e] * scale * (post ? w_post[e] + p.offset : 1.f) * g[e];
    } else if (post) {
#pragma unroll
      for (int e = 0; e < EPT; ++e) v[e] += x[e] * scale * (w_post[e] + p.offset);
    } else {
#pragma unroll
      for (int e = 0; e < EPT; ++e) v[e] += x[e] * scale;
    }
    if (p.out != nullptr)
      store_row<R, VEC, EPT>(static_cast<R*>(p.out) + static_cast<long long>(t) * p.ld_out, c, v);
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < EPT; ++e) q[0] += v[e] * v[e];
    const int next = slot + 1 == p.slots ? 0 : slot + 1;
    const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
    if (ahead && t + step < p.T) q[1] = take_y(t + step, next, next_phase);
    // behind this barrier every thread has its part of the slot
    group_sum<2>(q, p.tpr, 1 + group, tid, red, parity);
    if (tid == 0 && t + p.slots * step < p.T) ring.fill(slot, t + p.slots * step);
    slot = next;
    phase = next_phase;
    sq = q[1];
    if (pre) {
      const float f = rsqrtf(q[0] * inv_h + p.eps);
#pragma unroll
      for (int e = 0; e < EPT; ++e) v[e] *= f * (w_pre[e] + p.offset);
      store_row<A, VEC, EPT>(static_cast<A*>(p.h) + static_cast<long long>(t) * p.ld_h, c, v);
    }
  }
}

// Adds a thread's column sums of all groups of the CTA (in group order, through
// the row slots, which are free by then) and writes the CTA's partial row.
template <int VEC, int EPT>
__device__ __forceinline__ void cta_columns(float* buf, float* dst, const Cols<VEC>& c, int group,
                                            int groups, const float (&v)[EPT]) {
  for (int g = 0; g < groups; ++g) {
    __syncthreads();
    if (g == group) {
#pragma unroll
      for (int e = 0; e < EPT; ++e)
        if (c.col(e) < c.H) {
          const int at = c.col(e);
          const float s = g == 0 ? v[e] : buf[at] + v[e];
          if (g + 1 == groups)
            dst[at] = s;
          else
            buf[at] = s;
        }
    }
  }
}

template <typename R, typename A, int VEC, int EPT, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) block_norm_backward_kernel(const NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const NormSmem L = norm_smem(p.slot_bytes, p.slots, p.groups);
  const int group = threadIdx.x / p.tpr, tid = threadIdx.x - group * p.tpr;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  float* red = reinterpret_cast<float*>(smem + L.red) + group * 2 * kSumFloats;
  Ring<R, A, true> ring;
  ring.base = smem + static_cast<uint32_t>(group * p.slots) * p.slot_bytes;
  ring.full = bars + group * p.slots;
  ring.p = &p;
  ring.bytes_r = static_cast<uint32_t>(p.H * sizeof(R));
  ring.bytes_a = static_cast<uint32_t>(p.H * sizeof(A));
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.groups * p.slots; ++i) mbar_init(bars + i, 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait_and_trigger();
  const int step = gridDim.x * p.groups;
  const int first = blockIdx.x + gridDim.x * group;
  if (tid == 0)
    for (int s = 0; s < p.slots; ++s)
      if (first + s * step < p.T) ring.fill(s, first + s * step);
  const Cols<VEC> c{tid, p.tpr, p.H};
  const bool post = p.w_post != nullptr, pre = p.w_pre != nullptr, branch = p.y != nullptr;
  const float inv_h = 1.f / static_cast<float>(p.H);
  float a_post[EPT], a_pre[EPT], a_gate[EPT];   // column sums of dw_post, dw_pre, dg
#pragma unroll
  for (int e = 0; e < EPT; ++e) a_post[e] = a_pre[e] = a_gate[e] = 0.f;
  Kept<A, VEC, EPT> w_post, w_pre;
  w_post.zero();
  w_pre.zero();
  if (post) w_post.load(static_cast<const A*>(p.w_post), c);
  if (pre) w_pre.load(static_cast<const A*>(p.w_pre), c);
  // Rows behind this one's sums: a slot is filled again behind the sums of the
  // next row, so three are needed for sum(y^2) to run a row ahead.
  const bool ahead = p.slots > 2;
  auto wait = [&](int sl, uint32_t ph) {
    if (!mbar_wait(ring.full + sl, ph, nullptr)) report(p.status, MOE_ERR_DEVICE_TIMEOUT);
  };
  auto y_at = [&](int t, int sl) {
    return reinterpret_cast<const A*>(ring.base + static_cast<uint32_t>(sl) * p.slot_bytes + p.pitch_r +
                                      (VEC == 1 ? skew(ring.y_row(t)) : 0));
  };
  auto squares = [&](int t, int sl) {
    Kept<A, VEC, EPT> y;
    y.load(y_at(t, sl), c);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) q += y[e] * y[e];
    return q;
  };
  int slot = 0, parity = 0, before = 0;
  uint32_t phase = 0;
  float sq = 0.f;                               // sum of squares of the row's y
  for (int t = first; t < p.T; t += step) {
    if (t == first || !ahead) {
      wait(slot, phase);
      float q[2] = {post ? squares(t, slot) : 0.f, 0.f};
      if (post) group_sum<2>(q, p.tpr, 1 + group, tid, red, parity);
      sq = q[0];
    }
    const float fy = post ? rsqrtf(sq * inv_h + p.eps) : 1.f;
    float tg = 1.f;                             // gate of the token
    if (p.gate == MOE_GATE_TOKEN) tg = to_f<A>(static_cast<const A*>(p.gate_p)[t]);
    const uint8_t* at = ring.base + static_cast<uint32_t>(slot) * p.slot_bytes;
    const R* s_r = reinterpret_cast<const R*>(at + (VEC == 1 ? skew(ring.r_row(t)) : 0));
    at += p.pitch_r + p.pitch_a;
    const A* s_g = nullptr;
    if (p.gate == MOE_GATE_FULL) {
      s_g = reinterpret_cast<const A*>(at + (VEC == 1 ? skew(ring.g_row(t)) : 0));
      at += p.pitch_a;
    } else if (p.gate == MOE_GATE_CHANNEL) {
      s_g = static_cast<const A*>(p.gate_p);
    }
    const R* s_do = reinterpret_cast<const R*>(at + (VEC == 1 ? skew(ring.dout_row(t)) : 0));
    at += p.pitch_r;
    const A* s_dh = reinterpret_cast<const A*>(at + (VEC == 1 ? skew(ring.dh_row(t)) : 0));

    // n = y rstd(y) and u = bs g n w_post (without the token's gate), element
    // by element again in both passes below
    Kept<A, VEC, EPT> y, g, dh;
    Kept<R, VEC, EPT> dr, r;
    y.zero();
    dr.zero();
    r.zero();
    dh.zero();
    if (branch) y.load(y_at(t, slot), c);
    if (s_g != nullptr) g.load(s_g, c);
    if (p.d_out != nullptr) dr.load(s_do, c);
    if (pre) {
      r.load(s_r, c);
      dh.load(s_dh, c);
    }
    const float su = p.bs * fy;
    auto u_of = [&](int e) {
      float u = y[e] * su;
      if (post) u *= w_post[e] + p.offset;
      if (s_g != nullptr) u *= g[e];
      return u;
    };
    // one round of sums for both norms: with m~ = r', d = dh w_pre,
    //   mean(d m) = f^2 sum(d m~) / H,  f = rstd(r')
    //   sum(D u) = sum(dr' u) + f sum(d u) - f mean sum(m~ u)
    float q[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const float u = u_of(e), m = p.rs * r[e] + tg * u, d = dh[e] * (w_pre[e] + p.offset);
      q[0] += m * m;
      q[1] += d * m;
      q[2] += dr[e] * u;
      q[3] += d * u;
      q[4] += m * u;
    }
    const int next = slot + 1 == p.slots ? 0 : slot + 1;
    const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
    if (ahead && t + step < p.T) {
      wait(next, next_phase);
      if (post) q[5] = squares(t + step, next);
    }
    // behind this barrier everyone is done with the row before
    group_sum<8>(q, p.tpr, 1 + group, tid, red, parity);
    if (ahead && tid == 0 && t != first && t + (p.slots - 1) * step < p.T)
      ring.fill(before, t + (p.slots - 1) * step);
    sq = q[5];
    const float f = pre ? rsqrtf(q[0] * inv_h + p.eps) : 0.f, mean_h = q[1] * inv_h * f * f;
    const float sum_u = q[2] + f * (q[3] - mean_h * q[4]);
    if (p.gate == MOE_GATE_TOKEN && tid == 0) static_cast<float*>(p.d_gate)[t] = sum_u;
    float D[EPT], o[EPT];                       // the whole gradient at r'
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const float m = p.rs * r[e] + tg * u_of(e);
      a_pre[e] += dh[e] * m * f;
      D[e] = dr[e] + f * (dh[e] * (w_pre[e] + p.offset) - m * mean_h);
      o[e] = p.rs * D[e];
    }
    store_row<R, VEC, EPT>(static_cast<R*>(p.out) + static_cast<long long>(t) * p.ld_out, c, o);
    if (branch) {
      if (s_g != nullptr) {
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
          o[e] = D[e] * y[e] * su;
          if (post) o[e] *= w_post[e] + p.offset;
          a_gate[e] += o[e];
          D[e] *= g[e];
        }
        if (p.gate == MOE_GATE_FULL)
          store_row<A, VEC, EPT>(static_cast<A*>(p.d_gate) + static_cast<long long>(t) * p.ld_g, c, o);
      }
      // sum(dz z) over the row is the token's gate times sum(D u)
      const float mean_y = sum_u * tg * inv_h, s = p.bs * tg;
      if (post) {
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
          const float dz = s * D[e], n = y[e] * fy;
          a_post[e] += dz * n;
          D[e] = fy * (dz * (w_post[e] + p.offset) - n * mean_y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < EPT; ++e) D[e] *= s;
      }
      store_row<A, VEC, EPT>(static_cast<A*>(p.h) + static_cast<long long>(t) * p.ld_h, c, D);
    }
    if (!ahead) {
      if (p.tpr == 32)
        __syncwarp();
      else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(p.tpr) : "memory");
      if (tid == 0 && t + p.slots * step < p.T) ring.fill(slot, t + p.slots * step);
    }
    before = slot;
    slot = next;
    phase = next_phase;
  }
  if (p.n_part > 0) {
    float* buf = reinterpret_cast<float*>(smem);
    float* dst = p.part + static_cast<size_t>(blockIdx.x) * p.n_part * p.H;
    if (post) {
      cta_columns<VEC, EPT>(buf, dst, c, group, p.groups, a_post);
      dst += p.H;
    }
    if (pre) {
      cta_columns<VEC, EPT>(buf, dst, c, group, p.groups, a_pre);
      dst += p.H;
    }
    if (p.gate == MOE_GATE_CHANNEL) cta_columns<VEC, EPT>(buf, dst, c, group, p.groups, a_gate);
  }
}

// Sums the CTAs' partial rows: 32 columns a CTA, eight slices of the parts,
// each in order, then the slices in order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ part, int parts,
                                                         int n_part, int H, float* o0, float* o1,
                                                         float* o2) {
  __shared__ float s[8][33];
  pdl_wait_and_trigger();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + lane;
  const long long width = static_cast<long long>(n_part) * H;
  float v = 0.f;
  if (col < width)
    for (int i = slice; i < parts; i += 8) v += part[i * width + col];
  s[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && col < width) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    const int which = static_cast<int>(col / H);
    float* o = which == 0 ? o0 : (which == 1 ? o1 : o2);
    o[col - static_cast<long long>(which) * H] = v;
  }
}

uint32_t row_pitch(int H, int es) { return (static_cast<uint32_t>(H) * es + 15u + 16u) & ~15u; }

// Threads a row, groups and slots: EPT elements a thread; as many groups as
// fit the threads of a CTA and the slots' memory, down to one group of one slot.
void shape_of(NormParams& p, int ept, int max_threads, int rows_r, int rows_a, int es_r, int es_a, int sm) {
  int tpr = (p.H + ept - 1) / ept;
  tpr = (tpr + 31) / 32 * 32;
  p.tpr = tpr;
  p.pitch_r = row_pitch(p.H, es_r);
  p.pitch_a = row_pitch(p.H, es_a);
  p.slot_bytes = (rows_r * p.pitch_r + rows_a * p.pitch_a + 127u) & ~127u;
  int groups = max_threads / tpr;
  if (tpr > 32 && groups > 15) groups = 15;     // one named barrier each
  // no more groups than there are rows for
  const int need = (p.T + sm - 1) / sm;
  if (groups > need) groups = need;
  while (groups > 1 && groups * 2 * p.slot_bytes > kSmemBudget) --groups;
  int slots = static_cast<int>(kSmemBudget / (groups * p.slot_bytes));
  slots = slots > 4 ? 4 : (slots < 1 ? 1 : slots);
  p.groups = groups;
  p.slots = slots;
}

template <typename R, typename A, int VEC, int EPT, int MAXT, bool BACK>
cudaError_t run(NormParams& p, int rows_r, int rows_a, int sm, int* grid, cudaStream_t s) {
  static bool done[64] = {false};
  shape_of(p, EPT, MAXT, rows_r, rows_a, sizeof(R), sizeof(A), sm);
  const int want = (p.T + p.groups - 1) / p.groups;
  *grid = want < sm ? want : sm;
  const uint32_t smem = norm_smem(p.slot_bytes, p.slots, p.groups).total;
  auto go = [&](auto k) {
    const cudaError_t e = set_smem_once(k, 227 * 1024, done);
    return e != cudaSuccess ? e : launch_pdl(k, dim3(*grid), dim3(p.tpr * p.groups), smem, s, p);
  };
  if constexpr (BACK)
    return go(block_norm_backward_kernel<R, A, VEC, EPT, MAXT>);
  else
    return go(block_norm_kernel<R, A, VEC, EPT, MAXT>);
}

// Elements a thread and threads a CTA.  The backward pass holds three column
// sums per element: 512 threads have the registers for it (with 1024 it spilled
// and took three times as long).  Forward, 16 elements from 1024 columns up, so
// that two or more rows are at work on an SM and one's sums run under another's.
template <typename R, typename A, int VEC>
cudaError_t pick(NormParams& p, bool back, int rows_r, int rows_a, int sm, int* grid, cudaStream_t s) {
  if (back) {
    if (p.H <= 8 * 512) return run<R, A, VEC, 8, 512, true>(p, rows_r, rows_a, sm, grid, s);
    if (p.H <= 16 * 512) return run<R, A, VEC, 16, 512, true>(p, rows_r, rows_a, sm, grid, s);
    return run<R, A, VEC, 32, 512, true>(p, rows_r, rows_a, sm, grid, s);
  }
  if (p.H <= 1024) return run<R, A, VEC, 8, 1024, false>(p, rows_r, rows_a, sm, grid, s);
  if (p.H <= 16 * 896) return run<R, A, VEC, 16, 896, false>(p, rows_r, rows_a, sm, grid, s);
  return run<R, A, VEC, 16, 1024, false>(p, rows_r, rows_a, sm, grid, s);
}

template <typename R, typename A>
cudaError_t pick_vec(NormParams& p, bool back, bool vec, int rows_r, int rows_a, int sm, int* grid,
                     cudaStream_t s) {
  return vec ? pick<R, A, 8>(p, back, rows_r, rows_a, sm, grid, s)
             : pick<R, A, 1>(p, back, rows_r, rows_a, sm, grid, s);
}

}  // namespace

bool block_norm_fits(int H, bool residual_f32, bool act_f32, bool full_gate, bool back) {
  const uint32_t r = row_pitch(H, residual_f32 ? 4 : 2), a = row_pitch(H, act_f32 ? 4 : 2);
  const uint32_t rows_r = back ? 2 : 1, rows_a = (back ? 2 : 1) + (full_gate ? 1 : 0);
  return rows_r * r + rows_a * a + 128 <= kSmemBudget;
}

size_t block_norm_part_bytes(int T, int H, int n_part) {
  const size_t ctas = T < kNormMaxCtas ? (T < 1 ? 1 : T) : kNormMaxCtas;
  return ctas * n_part * static_cast<size_t>(H) * 4;
}

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s) {
  NormParams p{};
  p.T = a.T;
  p.H = a.H;
  p.gate = a.gate_kind;
  p.eps = a.eps;
  p.offset = a.weight_offset;
  p.rs = a.residual_scale;
  p.bs = a.branch_scale;
  p.r = a.residual;
  p.y = a.branch;
  p.gate_p = a.gate;
  p.w_post = a.branch != nullptr ? a.w_post : nullptr;
  p.w_pre = a.w_pre;
  p.ld_r = a.ld_residual;
  p.ld_y = a.ld_branch;
  p.ld_g = a.ld_gate;
  p.ld_out = a.ld_out;
  p.ld_h = a.ld_h;
  p.out = a.out;
  p.h = a.h;
  p.d_out = a.d_out;
  p.d_h = a.d_h;
  p.ld_dout = a.ld_dout;
  p.ld_dh = a.ld_dh;
  p.d_gate = a.d_gate;
  p.part = a.part;
  p.status = a.status;
  const int es_r = a.residual_f32 ? 4 : 2, es_a = a.act_f32 ? 4 : 2;
  auto ok16 = [](const void* q, long long ld, int es) {
    return q == nullptr || ((reinterpret_cast<uintptr_t>(q) & 15u) == 0 && (ld * es) % 16 == 0);
  };
  const bool full = a.gate_kind == MOE_GATE_FULL, chan = a.gate_kind == MOE_GATE_CHANNEL;
  const bool vec = a.H % 8 == 0 && ok16(a.residual, a.ld_residual, es_r) &&
                   ok16(a.branch, a.ld_branch, es_a) && ok16(a.out, a.ld_out, es_r) &&
                   ok16(a.h, a.ld_h, es_a) && ok16(a.w_post, 0, es_a) && ok16(a.w_pre, 0, es_a) &&
                   (!full || (ok16(a.gate, a.ld_gate, es_a) && ok16(a.d_gate, a.ld_gate, es_a))) &&
                   (!chan || ok16(a.gate, 0, es_a)) && ok16(a.d_out, a.ld_dout, es_r) &&
                   ok16(a.d_h, a.ld_dh, es_a);
  const int sm = a.sm_count < 1 ? 1 : (a.sm_count < kNormMaxCtas ? a.sm_count : kNormMaxCtas);
  p.n_part = 0;
  float* o[3] = {nullptr, nullptr, nullptr};
  if (a.back) {
    // without tokens the branch may be null, and its weight's gradient is still 0
    if (p.w_post != nullptr || (a.T == 0 && a.w_post != nullptr)) o[p.n_part++] = a.d_w_post;
    if (p.w_pre != nullptr) o[p.n_part++] = a.d_w_pre;
    if (chan) o[p.n_part++] = static_cast<float*>(a.d_gate);
  }
  if (a.T == 0) {
    for (int i = 0; i < p.n_part; ++i) {
      const cudaError_t e = cudaMemsetAsync(o[i], 0, sizeof(float) * a.H, s);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  const int rows_r = a.back ? 2 : 1, rows_a = (a.back ? 2 : 1) + (full ? 1 : 0);
  int grid = 1;
  cudaError_t e;
  if (a.residual_f32 && a.act_f32)
    e = pick_vec<float, float>(p, a.back, vec, rows_r, rows_a, sm, &grid, s);
  else if (a.residual_f32)
    e = pick_vec<float, __nv_bfloat16>(p, a.back, vec, rows_r, rows_a, sm, &grid, s);
  else
    e = pick_vec<__nv_bfloat16, __nv_bfloat16>(p, a.back, vec, rows_r, rows_a, sm, &grid, s);
  if (e != cudaSuccess || p.n_part == 0) return e;
  const long long width = static_cast<long long>(p.n_part) * a.H;
  return launch_pdl(column_sum_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(256), 0,
                    s, static_cast<const float*>(a.part), grid, p.n_part, a.H, o[0], o[1], o[2]);
}

}  // namespace moe
