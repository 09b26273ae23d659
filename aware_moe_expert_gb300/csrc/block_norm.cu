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
// would have had to store.
//
// Bound: memory.  A group of TPR threads owns a row, EPT elements a thread, and
// walks over rows with a ring of row slots that bulk copies fill ahead, so the
// loads of the next rows run under the two (three backward) row sums of this
// one.  Rows of any alignment are copied as the 16-byte granules around them.
// Sums and everything between load and store are fp32; each output is rounded
// once.
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kMaxThreads = 1024;
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

// Sums N values over the group's threads; every thread gets the sums.  `red`
// holds one buffer per parity: a buffer is written again only two sums later,
// behind the barrier of the sum between, which follows everyone's reads.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int tpr, int bar, int tid, float* red,
                                          int& parity) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  if (tpr == 32) {
    __syncwarp();
    return;
  }
  float* buf = red + parity * 64;
  parity ^= 1;
  const int warp = tid >> 5, nw = tpr >> 5;
  if ((tid & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 32 + warp] = v[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = (tid & 31) < nw ? buf[i * 32 + (tid & 31)] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    v[i] = t;
  }
}

// Shared memory: [groups][slots] row slots, then the sum buffers, then barriers.
struct NormSmem {
  uint32_t red, bars, total;
};
__host__ __device__ inline NormSmem norm_smem(uint32_t slot_bytes, int slots, int groups) {
  NormSmem o;
  uint32_t b = slot_bytes * static_cast<uint32_t>(slots) * static_cast<uint32_t>(groups);
  o.red = b;
  b += static_cast<uint32_t>(groups) * 128 * 4;
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

template <typename R, typename A, int VEC, int EPT>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const NormSmem L = norm_smem(p.slot_bytes, p.slots, p.groups);
  const int group = threadIdx.x / p.tpr, tid = threadIdx.x - group * p.tpr;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  float* red = reinterpret_cast<float*>(smem + L.red) + group * 128;
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
  float w_post[EPT], w_pre[EPT], gate[EPT];
  const bool post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  if (post) load_row<A, VEC, EPT>(static_cast<const A*>(p.w_post), c, w_post);
  if (pre) load_row<A, VEC, EPT>(static_cast<const A*>(p.w_pre), c, w_pre);
  if (p.gate == MOE_GATE_CHANNEL) load_row<A, VEC, EPT>(static_cast<const A*>(p.gate_p), c, gate);
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    w_post[e] = post ? w_post[e] + p.offset : 1.f;
    w_pre[e] = pre ? w_pre[e] + p.offset : 1.f;
    if (p.gate == MOE_GATE_CHANNEL) w_post[e] *= gate[e];
    w_post[e] *= p.bs;
  }
  const float inv_h = 1.f / static_cast<float>(p.H);
  int slot = 0, parity = 0;
  uint32_t phase = 0;
  for (int t = first; t < p.T; t += step) {
    float tg = 1.f;
    if (p.gate == MOE_GATE_TOKEN) tg = to_f<A>(static_cast<const A*>(p.gate_p)[t]);
    if (!mbar_wait(ring.full + slot, phase, nullptr)) report(p.status, MOE_ERR_DEVICE_TIMEOUT);
    const uint8_t* at = ring.base + static_cast<uint32_t>(slot) * p.slot_bytes;
    float v[EPT], x[EPT];
    load_row<R, VEC, EPT>(reinterpret_cast<const R*>(at + (VEC == 1 ? skew(ring.r_row(t)) : 0)), c, v);
    at += p.pitch_r;
    float q[1] = {0.f};
    if (p.y != nullptr) {
      load_row<A, VEC, EPT>(reinterpret_cast<const A*>(at + (VEC == 1 ? skew(ring.y_row(t)) : 0)), c, x);
#pragma unroll
      for (int e = 0; e < EPT; ++e) q[0] += x[e] * x[e];
    }
    at += p.pitch_a;
    if (p.gate == MOE_GATE_FULL)
      load_row<A, VEC, EPT>(reinterpret_cast<const A*>(at + (VEC == 1 ? skew(ring.g_row(t)) : 0)), c, gate);
    // every thread has its part of the slot behind this barrier
    group_sum<1>(q, p.tpr, 1 + group, tid, red, parity);
    if (tid == 0 && t + p.slots * step < p.T) ring.fill(slot, t + p.slots * step);
    if (++slot == p.slots) {
      slot = 0;
      phase ^= 1u;
    }
    if (p.y != nullptr) {
      const float f = (post ? rsqrtf(q[0] * inv_h + p.eps) : 1.f) * tg;
#pragma unroll
      for (int e = 0; e < EPT; ++e) {
        float z = x[e] * f * w_post[e];
        if (p.gate == MOE_GATE_FULL) z *= gate[e];
        v[e] = p.rs * v[e] + z;
      }
    } else {
#pragma unroll
      for (int e = 0; e < EPT; ++e) v[e] *= p.rs;
    }
    if (p.out != nullptr)
      store_row<R, VEC, EPT>(static_cast<R*>(p.out) + static_cast<long long>(t) * p.ld_out, c, v);
    if (pre) {
      q[0] = 0.f;
#pragma unroll
      for (int e = 0; e < EPT; ++e) q[0] += v[e] * v[e];
      group_sum<1>(q, p.tpr, 1 + group, tid, red, parity);
      const float f = rsqrtf(q[0] * inv_h + p.eps);
#pragma unroll
      for (int e = 0; e < EPT; ++e) v[e] *= f * w_pre[e];
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

template <typename R, typename A, int VEC, int EPT>
__global__ void __launch_bounds__(kMaxThreads) block_norm_backward_kernel(const NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const NormSmem L = norm_smem(p.slot_bytes, p.slots, p.groups);
  const int group = threadIdx.x / p.tpr, tid = threadIdx.x - group * p.tpr;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  float* red = reinterpret_cast<float*>(smem + L.red) + group * 128;
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
  const bool post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  const float inv_h = 1.f / static_cast<float>(p.H);
  float a_post[EPT], a_pre[EPT], a_gate[EPT];   // column sums of dw_post, dw_pre, dg
#pragma unroll
  for (int e = 0; e < EPT; ++e) a_post[e] = a_pre[e] = a_gate[e] = 0.f;
  int slot = 0, parity = 0;
  uint32_t phase = 0;
  for (int t = first; t < p.T; t += step) {
    float tg = 1.f;
    if (p.gate == MOE_GATE_TOKEN) tg = to_f<A>(static_cast<const A*>(p.gate_p)[t]);
    if (!mbar_wait(ring.full + slot, phase, nullptr)) report(p.status, MOE_ERR_DEVICE_TIMEOUT);
    const uint8_t* at = ring.base + static_cast<uint32_t>(slot) * p.slot_bytes;
    const R* s_r = reinterpret_cast<const R*>(at + (VEC == 1 ? skew(ring.r_row(t)) : 0));
    at += p.pitch_r;
    const A* s_y = reinterpret_cast<const A*>(at + (VEC == 1 ? skew(ring.y_row(t)) : 0));
    at += p.pitch_a;
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

    float n[EPT], w[EPT], z[EPT], d[EPT];   // n = y rstd(y), z = n w_post
    float fy = 1.f;
    if (p.y != nullptr) {
      load_row<A, VEC, EPT>(s_y, c, n);
      if (post) {
        float q[1] = {0.f};
#pragma unroll
        for (int e = 0; e < EPT; ++e) q[0] += n[e] * n[e];
        group_sum<1>(q, p.tpr, 1 + group, tid, red, parity);
        fy = rsqrtf(q[0] * inv_h + p.eps);
      }
    } else {
#pragma unroll
      for (int e = 0; e < EPT; ++e) n[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      n[e] *= fy;
      z[e] = n[e];
    }
    if (post) {
      load_row<A, VEC, EPT>(static_cast<const A*>(p.w_post), c, w);
#pragma unroll
      for (int e = 0; e < EPT; ++e) z[e] *= w[e] + p.offset;
    }
    if (p.d_out != nullptr) {
      load_row<R, VEC, EPT>(s_do, c, d);
    } else {
#pragma unroll
      for (int e = 0; e < EPT; ++e) d[e] = 0.f;
    }
    if (pre) {
      float m[EPT], dm[EPT];
      load_row<R, VEC, EPT>(s_r, c, m);
      if (s_g != nullptr) {
        load_row<A, VEC, EPT>(s_g, c, dm);
#pragma unroll
        for (int e = 0; e < EPT; ++e) m[e] = p.rs * m[e] + p.bs * dm[e] * z[e];
      } else {
#pragma unroll
        for (int e = 0; e < EPT; ++e) m[e] = p.rs * m[e] + p.bs * tg * z[e];
      }
      load_row<A, VEC, EPT>(s_dh, c, dm);
      load_row<A, VEC, EPT>(static_cast<const A*>(p.w_pre), c, w);
      float q[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < EPT; ++e) {
        q[0] += m[e] * m[e];
        q[1] += dm[e] * (w[e] + p.offset) * m[e];
      }
      group_sum<2>(q, p.tpr, 1 + group, tid, red, parity);
      const float f = rsqrtf(q[0] * inv_h + p.eps);
      const float mean = q[1] * inv_h * f * f;   // mean(dh w m~) rstd^2 with m~ = r'
#pragma unroll
      for (int e = 0; e < EPT; ++e) {
        a_pre[e] += dm[e] * m[e] * f;
        d[e] += f * (dm[e] * (w[e] + p.offset) - m[e] * mean);
      }
    }
    {
      float dr[EPT];
#pragma unroll
      for (int e = 0; e < EPT; ++e) dr[e] = p.rs * d[e];
      store_row<R, VEC, EPT>(static_cast<R*>(p.out) + static_cast<long long>(t) * p.ld_out, c, dr);
    }
    if (p.y != nullptr) {
#pragma unroll
      for (int e = 0; e < EPT; ++e) d[e] *= p.bs;
      float q[2] = {0.f, 0.f};   // sum d z (token gate), sum dz w n
      if (s_g != nullptr) {
        float g[EPT];
        load_row<A, VEC, EPT>(s_g, c, g);
        if (p.gate == MOE_GATE_FULL) {
          float dg[EPT];
#pragma unroll
          for (int e = 0; e < EPT; ++e) dg[e] = d[e] * z[e];
          store_row<A, VEC, EPT>(static_cast<A*>(p.d_gate) + static_cast<long long>(t) * p.ld_g, c, dg);
        } else {
#pragma unroll
          for (int e = 0; e < EPT; ++e) a_gate[e] += d[e] * z[e];
        }
#pragma unroll
        for (int e = 0; e < EPT; ++e) d[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < EPT; ++e) q[0] += d[e] * z[e];
      group_sum<1>(reinterpret_cast<float(&)[1]>(q[0]), p.tpr, 1 + group, tid, red, parity);
      // token gate: d is without g, so the sum is dg itself and g times it is sum dz z
      if (p.gate == MOE_GATE_TOKEN && tid == 0) static_cast<float*>(p.d_gate)[t] = q[0];
      const float mean = q[0] * tg * inv_h;
      float dy[EPT];
      if (post) {
        load_row<A, VEC, EPT>(static_cast<const A*>(p.w_post), c, w);
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
          const float dz = d[e] * tg;
          a_post[e] += dz * n[e];
          dy[e] = fy * (dz * (w[e] + p.offset) - n[e] * mean);
        }
      } else {
#pragma unroll
        for (int e = 0; e < EPT; ++e) dy[e] = d[e] * tg;
      }
      store_row<A, VEC, EPT>(static_cast<A*>(p.h) + static_cast<long long>(t) * p.ld_h, c, dy);
    }
    // everyone is done with the slot
    if (p.tpr == 32)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(p.tpr) : "memory");
    if (tid == 0 && t + p.slots * step < p.T) ring.fill(slot, t + p.slots * step);
    if (++slot == p.slots) {
      slot = 0;
      phase ^= 1u;
    }
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
// fit 1024 threads and the slots' memory, down to one group of one slot.
void shape_of(NormParams& p, int ept, int rows_r, int rows_a, int es_r, int es_a, int sm) {
  int tpr = (p.H + ept - 1) / ept;
  tpr = (tpr + 31) / 32 * 32;
  p.tpr = tpr;
  p.pitch_r = row_pitch(p.H, es_r);
  p.pitch_a = row_pitch(p.H, es_a);
  p.slot_bytes = (rows_r * p.pitch_r + rows_a * p.pitch_a + 127u) & ~127u;
  int groups = kMaxThreads / tpr;
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

template <typename R, typename A, int VEC, int EPT>
cudaError_t run(const NormParams& p, bool back, int grid, cudaStream_t s) {
  static bool done[64] = {false}, done_b[64] = {false};
  const uint32_t smem = norm_smem(p.slot_bytes, p.slots, p.groups).total;
  const dim3 g(grid), b(p.tpr * p.groups);
  if (back) {
    auto k = block_norm_backward_kernel<R, A, VEC, EPT>;
    const cudaError_t e = set_smem_once(k, 227 * 1024, done_b);
    return e != cudaSuccess ? e : launch_pdl(k, g, b, smem, s, p);
  }
  auto k = block_norm_kernel<R, A, VEC, EPT>;
  const cudaError_t e = set_smem_once(k, 227 * 1024, done);
  return e != cudaSuccess ? e : launch_pdl(k, g, b, smem, s, p);
}

template <typename R, typename A>
cudaError_t pick(NormParams& p, bool back, bool vec, int rows_r, int rows_a, int sm, int* grid,
                 cudaStream_t s) {
  const int ept = p.H <= 8 * kMaxThreads ? 8 : 16;
  shape_of(p, ept, rows_r, rows_a, sizeof(R), sizeof(A), sm);
  const int want = (p.T + p.groups - 1) / p.groups;
  *grid = want < sm ? want : sm;
  if (ept == 8)
    return vec ? run<R, A, 8, 8>(p, back, *grid, s) : run<R, A, 1, 8>(p, back, *grid, s);
  return vec ? run<R, A, 8, 16>(p, back, *grid, s) : run<R, A, 1, 16>(p, back, *grid, s);
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
    e = pick<float, float>(p, a.back, vec, rows_r, rows_a, sm, &grid, s);
  else if (a.residual_f32)
    e = pick<float, __nv_bfloat16>(p, a.back, vec, rows_r, rows_a, sm, &grid, s);
  else
    e = pick<__nv_bfloat16, __nv_bfloat16>(p, a.back, vec, rows_r, rows_a, sm, &grid, s);
  if (e != cudaSuccess || p.n_part == 0) return e;
  const long long width = static_cast<long long>(p.n_part) * a.H;
  return launch_pdl(column_sum_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(256), 0,
                    s, static_cast<const float*>(a.part), grid, p.n_part, a.H, o[0], o[1], o[2]);
}

}  // namespace moe
