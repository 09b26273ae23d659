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
// the next row is taken with the sums of this one.
// Rows need no alignment: they are copied as the 16-byte granules around them,
// and a thread's eight columns are the ones of an aligned 16-byte (32-byte for
// fp32) piece of memory.  A group's rows are a multiple of eight apart, so all of them
// start at the same place of such a piece, and a thread keeps its columns,
// weights and column sums.  Only tensors whose rows start at different places
// from each other take one column at a time.
// Sums and everything between load and store are fp32; each output is rounded
// once.
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr uint32_t kSmemBudget = 200 * 1024;   // row slots
constexpr uint32_t kSmemMost = 227 * 1024;     // and with the sum buffers and barriers

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// How a thread's EPT elements lie in a row of H columns.
enum Vec {
  kOne = 1,      // columns tid + e tpr, one at a time
  kPieces = 8,   // whole pieces of eight columns
  kSkewed = 9    // pieces of eight columns, the first of which begins `skew` before the row
};

template <int VEC, int EPT>
struct Cols {
  int tid, tpr, H, skew;
  uint32_t mask[VEC == kSkewed ? (EPT + 31) / 32 : 1];   // kSkewed: bit e: element e is in the row
  uint32_t half[VEC == kSkewed ? EPT / 2 : 1];           // and the same over two bf16
  __device__ __forceinline__ Cols(int tid_, int tpr_, int H_, int skew_)
      : tid(tid_), tpr(tpr_), H(H_), skew(skew_) {
    if constexpr (VEC == kSkewed) {
#pragma unroll
      for (int i = 0; i < (EPT + 31) / 32; ++i) mask[i] = 0u;
#pragma unroll
      for (int e = 0; e < EPT; ++e)
        if (static_cast<unsigned>(col(e)) < static_cast<unsigned>(H)) mask[e / 32] |= 1u << (e % 32);
#pragma unroll
      for (int e = 0; e < EPT; e += 2) half[e / 2] = (in(e) ? 0xffffu : 0u) | (in(e + 1) ? 0xffff0000u : 0u);
    }
  }
  // first column of piece v, and its place from the first piece's start
  __device__ __forceinline__ int place(int v) const { return (tid + v * tpr) * 8; }
  __device__ __forceinline__ int first(int v) const { return place(v) - (VEC == kSkewed ? skew : 0); }
  __device__ __forceinline__ int col(int e) const {
    return VEC == kOne ? tid + e * tpr : first(e / 8) + e % 8;
  }
  __device__ __forceinline__ bool in(int e) const {
    if constexpr (VEC == kSkewed) return mask[e / 32] >> (e % 32) & 1u;
    return static_cast<unsigned>(col(e)) < static_cast<unsigned>(H);
  }
  // any of piece v is in the row; all of it is
  __device__ __forceinline__ bool some(int v) const { return first(v) < H; }
  __device__ __forceinline__ bool whole(int v) const {
    if constexpr (VEC == kSkewed) return (mask[v / 4] >> (v % 4 * 8) & 255u) == 255u;
    return some(v);
  }
};

// A thread's elements of a row as they are in memory (bf16 two to a register);
// those outside the row are 0.  `p`: the row's column -skew (kOne: column 0).
template <typename T, int VEC, int EPT>
struct Row;
template <int VEC, int EPT>
struct Row<float, VEC, EPT> {
  float v[EPT];
  __device__ __forceinline__ void load(const float* p, const Cols<VEC, EPT>& c) {
    if constexpr (VEC == kOne) {
#pragma unroll
      for (int e = 0; e < EPT; ++e) v[e] = c.in(e) ? p[c.col(e)] : 0.f;
    } else {
#pragma unroll
      for (int e = 0; e < EPT; e += 4) {
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c.some(e / 8)) q = *reinterpret_cast<const float4*>(p + c.place(e / 8) + e % 8);
        v[e] = q.x;
        v[e + 1] = q.y;
        v[e + 2] = q.z;
        v[e + 3] = q.w;
      }
      if constexpr (VEC == kSkewed) {
#pragma unroll
        for (int e = 0; e < EPT; ++e) v[e] = c.in(e) ? v[e] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void set(int e, float x) { v[e] = x; }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < EPT; ++e) v[e] = 0.f;
  }
  __device__ __forceinline__ float2 pair(int i) const { return make_float2(v[2 * i], v[2 * i + 1]); }
};
template <int VEC, int EPT>
struct Row<__nv_bfloat16, VEC, EPT> {
  uint32_t v[EPT / 2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const Cols<VEC, EPT>& c) {
    if constexpr (VEC == kOne) {
      const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
      for (int e = 0; e < EPT; e += 2)
        v[e / 2] = (c.in(e) ? u[c.col(e)] : 0u) |
                   (c.in(e + 1) ? static_cast<uint32_t>(u[c.col(e + 1)]) << 16 : 0u);
    } else {
#pragma unroll
      for (int e = 0; e < EPT; e += 8) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (c.some(e / 8)) q = *reinterpret_cast<const uint4*>(p + c.place(e / 8));
        v[e / 2] = q.x;
        v[e / 2 + 1] = q.y;
        v[e / 2 + 2] = q.z;
        v[e / 2 + 3] = q.w;
      }
      if constexpr (VEC == kSkewed) {
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) v[i] &= c.half[i];
      }
    }
  }
  __device__ __forceinline__ void set(int e, float x) {    // x: a bf16 value
    const uint32_t b = __float_as_uint(x) >> 16;
    v[e / 2] = (e & 1) ? (v[e / 2] & 0xffffu) | (b << 16) : (v[e / 2] & 0xffff0000u) | b;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < EPT / 2; ++e) v[e] = 0u;
  }
  __device__ __forceinline__ float2 pair(int i) const { return make_float2(bf16lo(v[i]), bf16hi(v[i])); }
};

// Two elements at a time: the SM's packed fp32 instructions halve the
// arithmetic's share of the issue slots, which bound the backward pass.
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// Columns of a vector [H] that every row shares (any alignment).
template <typename T, int VEC, int EPT>
__device__ __forceinline__ void load_cols(const T* __restrict__ p, const Cols<VEC, EPT>& c,
                                          float2 (&v)[EPT / 2]) {
#pragma unroll
  for (int i = 0; i < EPT / 2; ++i)
    v[i] = make_float2(c.in(2 * i) ? to_f(p[c.col(2 * i)]) : 0.f,
                       c.in(2 * i + 1) ? to_f(p[c.col(2 * i + 1)]) : 0.f);
}

// `p`: the row's column 0.
template <typename T, int VEC, int EPT>
__device__ __forceinline__ void store_row(T* __restrict__ p, const Cols<VEC, EPT>& c,
                                          const float2 (&v)[EPT / 2]) {
  if constexpr (VEC == kOne) {
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) {
      if (c.in(2 * i)) p[c.col(2 * i)] = from_f<T>(v[i].x);
      if (c.in(2 * i + 1)) p[c.col(2 * i + 1)] = from_f<T>(v[i].y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < EPT; e += 8) {
      T* at = p + c.first(e / 8);
      const float2 &a = v[e / 2], &b = v[e / 2 + 1], &d = v[e / 2 + 2], &f = v[e / 2 + 3];
      if (c.whole(e / 8)) {
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<uint4*>(at) = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y),
                                                     pack_bf16x2(d.x, d.y), pack_bf16x2(f.x, f.y));
        } else {
          *reinterpret_cast<float4*>(at) = make_float4(a.x, a.y, b.x, b.y);
          *reinterpret_cast<float4*>(at + 4) = make_float4(d.x, d.y, f.x, f.y);
        }
      } else if constexpr (VEC == kSkewed) {
        // the row's first or last piece
        if (c.in(e)) at[0] = from_f<T>(a.x);
        if (c.in(e + 1)) at[1] = from_f<T>(a.y);
        if (c.in(e + 2)) at[2] = from_f<T>(b.x);
        if (c.in(e + 3)) at[3] = from_f<T>(b.y);
        if (c.in(e + 4)) at[4] = from_f<T>(d.x);
        if (c.in(e + 5)) at[5] = from_f<T>(d.y);
        if (c.in(e + 6)) at[6] = from_f<T>(f.x);
        if (c.in(e + 7)) at[7] = from_f<T>(f.y);
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

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
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
    // four warps' sums a load where few lanes share a value, which takes a `red`
    // that was cleared (backward, 8192 x 2048: 49 us, 51 one at a time; forward,
    // 16384 x 7168: 155 and 148)
    const float* from = buf + value * 32;
    const int l = lane % kLanes;
#pragma unroll
    for (int w = 0; w < 32; w += N == 8 ? 4 * kLanes : kLanes) {
      if (w >= nw) break;
      if constexpr (N == 8) {
        const float4 q = *reinterpret_cast<const float4*>(from + w + 4 * l);
        part += (q.x + q.y) + (q.z + q.w);
      } else {
        part += w < nw - l ? from[w + l] : 0.f;
      }
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) part += __shfl_xor_sync(kAll, part, off);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(kAll, part, i * (32 / N));
}

__device__ __noinline__ void wait_long(uint64_t* bar, uint32_t phase, int32_t* status) {
  if (!mbar_wait(bar, phase, nullptr)) report(status, MOE_ERR_DEVICE_TIMEOUT);
}

// Shared memory: [groups][slots] row slots, then the sum buffers, then barriers.
struct NormSmem {
  uint32_t red, bars, total;
};
// Two barriers a slot: full, and (forward) empty.
__host__ __device__ inline NormSmem norm_smem(uint32_t slot_bytes, int slots, int groups) {
  NormSmem o;
  uint32_t b = slot_bytes * static_cast<uint32_t>(slots) * static_cast<uint32_t>(groups);
  o.red = b;
  b += static_cast<uint32_t>(groups) * 2 * kSumFloats * 4;
  o.bars = b;
  b += static_cast<uint32_t>(groups * slots) * 16;
  o.total = b;
  return o;
}

// One group's ring.  A slot holds the rows r, y, [gate], [dr'], [dh] of a token,
// each as the 16-byte granules around it.  Pieces: column -skew lies at the
// start of its place; kOne: the granules do.
// Filling a slot is a chain of address arithmetic, and a thread of the group
// that did it alone held up the group's next sums for longer than the sums
// took.  Forward, a warp of its own does it, a lane for each group (Producer);
// backward, whose registers leave no room for one, the group's first warp, a
// lane for each tensor (Filler).
template <typename R, typename A, int VEC>
struct Ring {
  uint8_t* base;
  uint64_t* full;
  const NormParams* p;

  __device__ __forceinline__ Ring(const NormParams* q, uint8_t* smem, uint64_t* bars, int group)
      : base(smem + static_cast<uint32_t>(group * q->slots) * q->slot_bytes),
        full(bars + group * q->slots),
        p(q) {}
  // a row's place in a slot, as Row::load wants it
  template <typename T>
  __device__ __forceinline__ const T* place(int slot, uint32_t off, const void* q, int t, long long ld) const {
    off += static_cast<uint32_t>(slot) * p->slot_bytes;
    if (VEC == kOne)
      off += static_cast<uint32_t>(
          reinterpret_cast<uintptr_t>(static_cast<const T*>(q) + static_cast<long long>(t) * ld) & 15u);
    return reinterpret_cast<const T*>(base + off);
  }
  __device__ __forceinline__ void wait(int slot, uint32_t phase) const {
    if (!mbar_try_wait(full + slot, phase)) wait_long(full + slot, phase, p->status);
  }
};

// The rows of one tensor that a group copies.
template <int VEC>
struct RowStream {
  uintptr_t next = 0;           // the next row
  long long stride = 0;
  uint32_t bytes = 0, at = 0, before = 0;

  template <typename T>
  __device__ __forceinline__ void take(const NormParams& p, const void* q, long long ld, uint32_t place,
                                       int skew, int first, int step) {
    if (q == nullptr) return;
    next = reinterpret_cast<uintptr_t>(q) + static_cast<long long>(first) * ld * static_cast<long long>(sizeof(T));
    stride = static_cast<long long>(step) * ld * static_cast<long long>(sizeof(T));
    bytes = static_cast<uint32_t>(p.H) * sizeof(T);
    at = place;
    before = VEC == kOne ? 0u : static_cast<uint32_t>(skew) * sizeof(T);
  }
  __device__ __forceinline__ uintptr_t from() const { return next & ~static_cast<uintptr_t>(15); }
  __device__ __forceinline__ uint32_t size() const {
    return bytes != 0u ? static_cast<uint32_t>(((next + bytes + 15) & ~static_cast<uintptr_t>(15)) - from()) : 0u;
  }
  __device__ __forceinline__ void copy(uint32_t slot, uint64_t* full) {
    if (bytes == 0u) return;
    const uint32_t skip = VEC == kOne ? 0u : static_cast<uint32_t>(from() - (next - before));
    bulk_load(slot + at + skip, reinterpret_cast<const void*>(from()), size(), full);
    next += stride;
  }
};

// A lane of the forward pass's producer warp: every row of its group, a slot as
// soon as it is free.
template <typename R, typename A, int VEC>
__device__ __forceinline__ void produce(const Ring<R, A, VEC>& ring, uint64_t* empty, int skew, int first,
                                        int step) {
  const NormParams& p = *ring.p;
  RowStream<VEC> r, y, g;
  r.template take<R>(p, p.r, p.ld_r, 0u, skew, first, step);
  y.template take<A>(p, p.y, p.ld_y, p.pitch_r, skew, first, step);
  if (p.gate == MOE_GATE_FULL)
    g.template take<A>(p, p.gate_p, p.ld_g, p.pitch_r + p.pitch_a, skew, first, step);
  uint32_t phase = 1;
  int slot = 0;
  for (int t = first; t < p.T; t += step) {
    if (!mbar_wait(empty + slot, phase, nullptr)) {
      report(p.status, MOE_ERR_DEVICE_TIMEOUT);
      return;
    }
    const uint32_t to = smem_u32(ring.base) + static_cast<uint32_t>(slot) * p.slot_bytes;
    mbar_expect_tx(ring.full + slot, r.size() + y.size() + g.size());
    r.copy(to, ring.full + slot);
    y.copy(to, ring.full + slot);
    g.copy(to, ring.full + slot);
    if (++slot == p.slots) {
      slot = 0;
      phase ^= 1u;
    }
  }
}

// The backward pass's: lane i of the group's first warp has tensor i.
template <typename R, typename A, int VEC>
struct Filler {
  RowStream<VEC> s;
  int left;                     // rows still to copy

  __device__ __forceinline__ Filler(const NormParams& p, int skew, int first, int step, int lane)
      : left(first < p.T ? (p.T - 1 - first) / step + 1 : 0) {
    const bool gate = p.gate == MOE_GATE_FULL;
    const uint32_t o_gate = p.pitch_r + p.pitch_a, o_do = o_gate + (gate ? p.pitch_a : 0u);
    if (lane == 0) s.template take<R>(p, p.r, p.ld_r, 0u, skew, first, step);
    if (lane == 1) s.template take<A>(p, p.y, p.ld_y, p.pitch_r, skew, first, step);
    if (lane == 2 && gate) s.template take<A>(p, p.gate_p, p.ld_g, o_gate, skew, first, step);
    // (forward: null)
    if (lane == 3) s.template take<R>(p, p.d_out, p.ld_dout, o_do, skew, first, step);
    if (lane == 4) s.template take<A>(p, p.d_h, p.ld_dh, o_do + p.pitch_r, skew, first, step);
  }
  // the group's next row into `slot`
  __device__ __forceinline__ void fill(const Ring<R, A, VEC>& ring, int slot, int lane) {
    if (left <= 0) return;
    --left;
    const uint32_t total = __reduce_add_sync(0xffffffffu, s.size());
    if (lane == 0) mbar_expect_tx(ring.full + slot, total);
    __syncwarp();
    s.copy(smem_u32(ring.base) + static_cast<uint32_t>(slot) * ring.p->slot_bytes, ring.full + slot);
  }
};

// Columns of the first piece before a group's rows: the same for all of them,
// since the rows are gridDim.x * groups apart (a multiple of eight, or the
// group has one row).
template <int VEC>
__device__ __forceinline__ int skew_of(const NormParams& p, int first) {
  return VEC == kSkewed ? static_cast<int>((static_cast<long long>(first) * p.ld_r) & 7) : 0;
}

// MAXT threads in groups, and the producer warp.  SELF: groups of one warp fill
// their own slots (31 of them kept one producer warp too busy: 16384 x 256 took 12
// us, 9 without).
// Measured: 16384 x 7168 bf16 with both norms 148 us, 6.4 TB/s, 0.94 of a copy;
// two block sums a row (one between the norms) are what is left of it.  16384 x
// 4096, fp32 residual and a full gate 136 us.  One row of 7168: 3.3 us.
template <typename R, typename A, int VEC, int EPT, int MAXT, bool SELF>
__global__ void __launch_bounds__(MAXT + (SELF ? 0 : 32), 1) block_norm_kernel(const NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const NormSmem L = norm_smem(p.slot_bytes, p.slots, p.groups);
  const bool producer = threadIdx.x >= p.tpr * p.groups;
  const int group = producer ? threadIdx.x & 31 : threadIdx.x / p.tpr;
  const int tid = threadIdx.x - group * p.tpr;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  float* red = reinterpret_cast<float*>(smem + L.red) + group * 2 * kSumFloats;
  const int step = gridDim.x * p.groups;
  const int first = blockIdx.x + gridDim.x * group;
  const Ring<R, A, VEC> ring(&p, smem, bars, group);
  uint64_t* empty = bars + (p.groups + group) * p.slots;
  const int skew = skew_of<VEC>(p, first);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * p.groups * p.slots; ++i) mbar_init(bars + i, 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait_and_trigger();
  Filler<R, A, VEC> filler(p, skew, first, step, SELF ? tid : 32);
  if (SELF) {
    for (int i = 0; i < p.slots; ++i) filler.fill(ring, i, tid);
  } else if (producer) {
    if (group < p.groups) produce(ring, empty, skew, first, step);
    return;
  }
  const Cols<VEC, EPT> c(tid, p.tpr, p.H, skew);
  const bool post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  // the weights of the thread's columns as they are in memory
  Row<A, VEC, EPT> w1, w2, g;
  w1.zero();
  w2.zero();
  auto take = [&](Row<A, VEC, EPT>& w, const void* q) {
    if (VEC == kPieces && (reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
      w.load(static_cast<const A*>(q), c);
      return;
    }
#pragma unroll
    for (int e = 0; e < EPT; ++e)
      if (c.in(e)) w.set(e, to_f(static_cast<const A*>(q)[c.col(e)]));
  };
  if (post) take(w1, p.w_post);
  if (pre) take(w2, p.w_pre);
  const bool vector_gate = p.gate == MOE_GATE_FULL || p.gate == MOE_GATE_CHANNEL;
  if (p.gate == MOE_GATE_CHANNEL) {
    g.zero();
    take(g, p.gate_p);
  }
  const float off1 = post ? p.offset : 1.f;      // without a post-norm: weight 1
  const float inv_h = 1.f / static_cast<float>(p.H);
  const bool ahead = p.slots > 1;     // the next row is there while this one is at work
  int slot = 0, parity = 0;
  uint32_t phase = 0;
  Row<A, VEC, EPT> x;                 // y of the row
  x.zero();
  float sq = 0.f;                     // its sum of squares
  auto take_y = [&](int t, int sl, uint32_t ph) {
    ring.wait(sl, ph);
    float q = 0.f;
    if (p.y != nullptr) {
      x.load(ring.template place<A>(sl, p.pitch_r, p.y, t, p.ld_y), c);
      float2 a = two(0.f);
#pragma unroll
      for (int i = 0; i < EPT / 2; ++i) a = fma(x.pair(i), x.pair(i), a);
      q = a.x + a.y;
    }
    return q;
  };
  R* out = static_cast<R*>(p.out) + static_cast<long long>(first) * p.ld_out;
  A* h = static_cast<A*>(p.h) + static_cast<long long>(first) * p.ld_h;
  const long long out_step = static_cast<long long>(step) * p.ld_out, h_step = static_cast<long long>(step) * p.ld_h;
  for (int t = first; t < p.T; t += step) {
    if (t == first || !ahead) {
      float q[2] = {take_y(t, slot, phase), 0.f};
      group_sum<2>(q, p.tpr, 1 + group, tid, red, parity);
      sq = q[0];
    }
    float scale = p.bs;
    if (p.gate == MOE_GATE_TOKEN) scale *= to_f(static_cast<const A*>(p.gate_p)[t]);
    if (post) scale *= rsqrtf(sq * inv_h + p.eps);
    float2 v[EPT / 2];
    {
      Row<R, VEC, EPT> r;
      r.load(ring.template place<R>(slot, 0, p.r, t, p.ld_r), c);
#pragma unroll
      for (int i = 0; i < EPT / 2; ++i) v[i] = mul(two(p.rs), r.pair(i));
    }
    if (vector_gate) {
      if (p.gate == MOE_GATE_FULL)
        g.load(ring.template place<A>(slot, p.pitch_r + p.pitch_a, p.gate_p, t, p.ld_g), c);
#pragma unroll
      for (int i = 0; i < EPT / 2; ++i)
        v[i] = fma(mul(mul(x.pair(i), two(scale)), g.pair(i)), add(w1.pair(i), two(off1)), v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < EPT / 2; ++i)
        v[i] = fma(mul(x.pair(i), two(scale)), add(w1.pair(i), two(off1)), v[i]);
    }
    if (p.out != nullptr) store_row(out, c, v);
    out += out_step;
    float2 vv = two(0.f);
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) vv = fma(v[i], v[i], vv);
    float q[2] = {vv.x + vv.y, 0.f};
    const int next = slot + 1 == p.slots ? 0 : slot + 1;
    const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
    if (ahead && t + step < p.T) q[1] = take_y(t + step, next, next_phase);
    // behind this barrier every thread has its part of the slot
    group_sum<2>(q, p.tpr, 1 + group, tid, red, parity);
    if (SELF)
      filler.fill(ring, slot, tid);
    else if (tid == 0)
      mbar_arrive(empty + slot);
    slot = next;
    phase = next_phase;
    sq = q[1];
    if (pre) {
      const float f = rsqrtf(q[0] * inv_h + p.eps);
#pragma unroll
      for (int i = 0; i < EPT / 2; ++i) v[i] = mul(mul(v[i], two(f)), add(w2.pair(i), two(p.offset)));
      store_row(h, c, v);
      h += h_step;
    }
  }
}

// A CTA's column sums: the groups' through shared memory (the row slots, which
// are free by then), added in group order, to the CTA's partial row.
template <int VEC, int EPT>
__device__ __forceinline__ void cta_columns(float* buf, float* dst, const Cols<VEC, EPT>& c, int group,
                                            int groups, const float2 (&v)[EPT / 2]) {
  __syncthreads();
#pragma unroll
  for (int i = 0; i < EPT / 2; ++i) {
    if (c.in(2 * i)) buf[group * c.H + c.col(2 * i)] = v[i].x;
    if (c.in(2 * i + 1)) buf[group * c.H + c.col(2 * i + 1)] = v[i].y;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < c.H; i += blockDim.x) {
    float s = buf[i];
    for (int g = 1; g < groups; ++g) s += buf[g * c.H + i];
    dst[i] = s;
  }
}

// Bound: issue slots (about 510 warp instructions a row and warp at eight elements
// a thread) under the 16 warps whose registers hold the column sums.  8192 x 2048
// bf16 with a gate per token: 50 us with the column sums' launch, 4.0 TB/s; 7168
// columns 245 us: one row at a time, 16 elements a thread, and spills.
template <typename R, typename A, int VEC, int EPT, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) block_norm_backward_kernel(const NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const NormSmem L = norm_smem(p.slot_bytes, p.slots, p.groups);
  const int group = threadIdx.x / p.tpr, tid = threadIdx.x - group * p.tpr;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  float* red = reinterpret_cast<float*>(smem + L.red) + group * 2 * kSumFloats;
  const int step = gridDim.x * p.groups;
  const int first = blockIdx.x + gridDim.x * group;
  const Ring<R, A, VEC> ring(&p, smem, bars, group);
  const int skew = skew_of<VEC>(p, first);
  Filler<R, A, VEC> filler(p, skew, first, step, tid);
  // group_sum reads the sums of warps that do not exist
  for (int i = threadIdx.x; i < p.groups * 2 * kSumFloats; i += blockDim.x)
    reinterpret_cast<float*>(smem + L.red)[i] = 0.f;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.groups * p.slots; ++i) mbar_init(bars + i, 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait_and_trigger();
  if (tid < 32)
    for (int i = 0; i < p.slots; ++i) filler.fill(ring, i, tid);
  const Cols<VEC, EPT> c(tid, p.tpr, p.H, skew);
  const bool post = p.w_post != nullptr, pre = p.w_pre != nullptr, branch = p.y != nullptr;
  const bool full = p.gate == MOE_GATE_FULL, vector_gate = full || p.gate == MOE_GATE_CHANNEL;
  const float inv_h = 1.f / static_cast<float>(p.H);
  constexpr int P = EPT / 2;
  float2 a_post[P], a_pre[P], a_gate[P];        // column sums of dw_post / bs, dw_pre, dg
  float2 w1[P], w2[P];                          // bs w_post, w_pre
#pragma unroll
  for (int i = 0; i < P; ++i) a_post[i] = a_pre[i] = a_gate[i] = w1[i] = w2[i] = two(0.f);
  if (post) load_cols<A>(static_cast<const A*>(p.w_post), c, w1);
  if (pre) load_cols<A>(static_cast<const A*>(p.w_pre), c, w2);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    w1[i] = post ? mul(add(w1[i], two(p.offset)), two(p.bs)) : two(p.bs);
    w2[i] = add(w2[i], two(p.offset));
  }
  Row<A, VEC, EPT> g;
  g.zero();
  if (p.gate == MOE_GATE_CHANNEL) {
    float2 w[P];
    load_cols<A>(static_cast<const A*>(p.gate_p), c, w);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      g.set(2 * i, w[i].x);
      g.set(2 * i + 1, w[i].y);
    }
  }
  const bool ahead = p.slots > 1;
  auto squares = [&](int t, int sl) {
    Row<A, VEC, EPT> y;
    y.load(ring.template place<A>(sl, p.pitch_r, p.y, t, p.ld_y), c);
    float2 q = two(0.f);
#pragma unroll
    for (int i = 0; i < P; ++i) q = fma(y.pair(i), y.pair(i), q);
    return q.x + q.y;
  };
  int slot = 0, parity = 0;
  uint32_t phase = 0;
  float sq = 0.f;                               // sum of squares of the row's y
  R* out = static_cast<R*>(p.out) + static_cast<long long>(first) * p.ld_out;
  A* dy = static_cast<A*>(p.h) + static_cast<long long>(first) * p.ld_h;
  const long long out_step = static_cast<long long>(step) * p.ld_out, dy_step = static_cast<long long>(step) * p.ld_h;
  for (int t = first; t < p.T; t += step) {
    if (t == first || !ahead) {
      ring.wait(slot, phase);
      float q[2] = {post ? squares(t, slot) : 0.f, 0.f};
      if (post) group_sum<2>(q, p.tpr, 1 + group, tid, red, parity);
      sq = q[0];
    }
    const float fy = post ? rsqrtf(sq * inv_h + p.eps) : 1.f;
    float tg = 1.f;                             // gate of the token
    if (p.gate == MOE_GATE_TOKEN) tg = to_f(static_cast<const A*>(p.gate_p)[t]);
    uint32_t at = p.pitch_r + p.pitch_a;
    if (full) {
      g.load(ring.template place<A>(slot, at, p.gate_p, t, p.ld_g), c);
      at += p.pitch_a;
    }
    Row<A, VEC, EPT> dh;
    Row<R, VEC, EPT> dr;
    dr.zero();
    dh.zero();
    if (p.d_out != nullptr) dr.load(ring.template place<R>(slot, at, p.d_out, t, p.ld_dout), c);
    if (pre) dh.load(ring.template place<A>(slot, at + p.pitch_r, p.d_h, t, p.ld_dh), c);
    // n = y rstd(y), u = bs g n w_post (without the token's gate), m~ = r'
    float2 n[P], m[P];
    {
      Row<R, VEC, EPT> r;
      Row<A, VEC, EPT> y;
      y.zero();
      r.load(ring.template place<R>(slot, 0, p.r, t, p.ld_r), c);
      if (branch) y.load(ring.template place<A>(slot, p.pitch_r, p.y, t, p.ld_y), c);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        n[i] = mul(y.pair(i), two(fy));
        m[i] = mul(r.pair(i), two(p.rs));
      }
    }
    // one round of sums for both norms: with d = dh w_pre,
    //   mean(d m) = f^2 sum(d m~) / H,  f = rstd(r')
    //   sum(D u) = sum(dr' u) + f sum(d u) - f mean sum(m~ u)
    float2 s[5] = {two(0.f), two(0.f), two(0.f), two(0.f), two(0.f)};
    auto gather = [&](int i, float2 u) {
      m[i] = fma(two(tg), u, m[i]);
      const float2 d = mul(dh.pair(i), w2[i]);
      s[0] = fma(m[i], m[i], s[0]);
      s[1] = fma(d, m[i], s[1]);
      s[2] = fma(dr.pair(i), u, s[2]);
      s[3] = fma(d, u, s[3]);
      s[4] = fma(m[i], u, s[4]);
    };
    if (vector_gate) {
#pragma unroll
      for (int i = 0; i < P; ++i) gather(i, mul(mul(n[i], w1[i]), g.pair(i)));
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) gather(i, mul(n[i], w1[i]));
    }
    float q[8] = {s[0].x + s[0].y, s[1].x + s[1].y, s[2].x + s[2].y, s[3].x + s[3].y,
                  s[4].x + s[4].y, 0.f, 0.f, 0.f};
    const int next = slot + 1 == p.slots ? 0 : slot + 1;
    const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
    if (ahead && t + step < p.T) {
      ring.wait(next, next_phase);
      if (post) q[5] = squares(t + step, next);
    }
    // behind this barrier everyone has the row in registers
    group_sum<8>(q, p.tpr, 1 + group, tid, red, parity);
    if (tid < 32) filler.fill(ring, slot, tid);
    sq = q[5];
    const float f = pre ? rsqrtf(q[0] * inv_h + p.eps) : 0.f, mean_h = q[1] * inv_h * f * f;
    const float sum_u = q[2] + f * (q[3] - mean_h * q[4]), c2 = f * mean_h;
    if (p.gate == MOE_GATE_TOKEN && tid == 0) static_cast<float*>(p.d_gate)[t] = sum_u;
    float2 D[P], o[P];                          // the whole gradient at r'
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 h = dh.pair(i);
      a_pre[i] = fma(h, mul(m[i], two(f)), a_pre[i]);
      D[i] = fma(m[i], two(-c2), fma(mul(h, w2[i]), two(f), dr.pair(i)));
      o[i] = mul(D[i], two(p.rs));
    }
    store_row(out, c, o);
    out += out_step;
    if (branch) {
      if (vector_gate) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          o[i] = mul(D[i], mul(n[i], w1[i]));
          a_gate[i] = add(a_gate[i], o[i]);
          D[i] = mul(D[i], g.pair(i));
        }
        if (full) store_row(static_cast<A*>(p.d_gate) + static_cast<long long>(t) * p.ld_g, c, o);
      }
      // sum(dz z) over the row is the token's gate times sum(D u)
      const float c3 = post ? fy * sum_u * tg * inv_h : 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 dz = mul(D[i], two(tg));
        a_post[i] = fma(dz, n[i], a_post[i]);
        D[i] = fma(mul(dz, w1[i]), two(fy), mul(n[i], two(-c3)));
      }
      store_row(dy, c, D);
      dy += dy_step;
    }
    slot = next;
    phase = next_phase;
  }
  if (p.n_part > 0) {
    float* buf = reinterpret_cast<float*>(smem);
    float* dst = p.part + static_cast<size_t>(blockIdx.x) * p.n_part * p.H;
    if (post) {
#pragma unroll
      for (int i = 0; i < P; ++i) a_post[i] = mul(a_post[i], two(p.bs));
      cta_columns(buf, dst, c, group, p.groups, a_post);
      dst += p.H;
    }
    if (pre) {
      cta_columns(buf, dst, c, group, p.groups, a_pre);
      dst += p.H;
    }
    if (p.gate == MOE_GATE_CHANNEL) cta_columns(buf, dst, c, group, p.groups, a_gate);
  }
}

// Sums the CTAs' partial rows: 32 columns a CTA, 32 slices of the parts, each in
// order, then the slices in order.
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices) column_sum_kernel(const float* __restrict__ part, int parts,
                                                                  int n_part, int H, float* o0, float* o1,
                                                                  float* o2) {
  __shared__ float s[kSlices][33];
  pdl_wait_and_trigger();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + lane;
  const long long width = static_cast<long long>(n_part) * H;
  constexpr int kMost = (kNormMaxCtas + kSlices - 1) / kSlices;
  float w[kMost], v = 0.f;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int r = slice + i * kSlices;
    w[i] = col < width && r < parts ? part[r * width + col] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kMost; ++i) v += w[i];
  s[slice][lane] = v;
  __syncthreads();
  // warp w sums columns w: lane = slice
  v = s[lane][slice];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  const long long mine = static_cast<long long>(blockIdx.x) * 32 + slice;
  if (lane == 0 && mine < width) {
    const int which = static_cast<int>(mine / H);
    float* o = which == 0 ? o0 : (which == 1 ? o1 : o2);
    o[mine - static_cast<long long>(which) * H] = v;
  }
}

// 16 bytes of slack for the granules and 16 for an fp32 piece that begins
// before them.
uint32_t row_pitch(int H, int es) { return (static_cast<uint32_t>(H + 7) * es + 15u + 32u) & ~15u; }

// Columns a group's threads span: a skewed row may begin seven into its first piece.
int span(const NormParams& p, int vec) { return p.H + (vec == kSkewed ? 7 : 0); }

// Threads a row, groups and slots: EPT elements a thread; as many groups as
// fit the threads of a CTA and the slots' memory, down to one group of one slot.
void shape_of(NormParams& p, int vec, int ept, int max_threads, int rows_r, int rows_a, int es_r, int es_a, int sm) {
  int tpr = (span(p, vec) + ept - 1) / ept;
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
  // the sum buffers count, too: 2 KB a group (138 to 389 columns, fp32, 14 to 16
  // groups); a third or fourth slot goes before a group does
  while (norm_smem(p.slot_bytes, slots, groups).total > kSmemMost) {
    if (slots > 2 || groups == 1)
      --slots;
    else
      --groups;
  }
  p.groups = groups;
  p.slots = slots;
}

template <typename R, typename A, int VEC, int EPT, int MAXT, bool BACK, bool SELF = false>
cudaError_t run(NormParams& p, int rows_r, int rows_a, int sm, NormPlan* plan, cudaStream_t s) {
  static bool done[64] = {false};
  shape_of(p, VEC, EPT, MAXT, rows_r, rows_a, sizeof(R), sizeof(A), sm);
  // a group's rows are grid * groups apart: a multiple of eight if there are several
  const int want = (p.T + p.groups - 1) / p.groups, most = sm >= 8 ? sm / 8 * 8 : sm;
  plan->grid = want <= sm ? want : most;
  if (want > sm && most % 8 != 0 && VEC == kSkewed) return cudaErrorInvalidConfiguration;
  plan->groups = p.groups;
  plan->slots = p.slots;
  plan->smem = norm_smem(p.slot_bytes, p.slots, p.groups).total;
  if (plan->only) return cudaSuccess;
  auto go = [&](auto k) {
    const cudaError_t e = set_smem_once(k, static_cast<int>(kSmemMost), done);
    return e != cudaSuccess ? e
                            : launch_pdl(k, dim3(plan->grid), dim3(p.tpr * p.groups + (BACK || SELF ? 0 : 32)),
                                         plan->smem, s, p);
  };
  if constexpr (BACK)
    return go(block_norm_backward_kernel<R, A, VEC, EPT, MAXT>);
  else
    return go(block_norm_kernel<R, A, VEC, EPT, MAXT, SELF>);
}

// Elements a thread and threads a CTA: eight elements as long as the threads
// reach (16384 x 7168: 148 us, 16 elements in 896 threads 205).  The backward
// pass holds three column sums per element: 512 threads have the registers for
// it (8192 x 2048: 50 us, 1024 threads spill and take 86).  Wider rows spill on both
// sides of these rules.  Forward, 16384 x 8192, 8192 x 12288 and 4096 x 16384: 239, 231
// and 130 us; 16 elements in 992 threads as far as they reach 414 and 211, 40 in 512
// threads 405, 324 and 195.  Backward, 8192 x 7168 and 8192: 245 and 260 us with 16
// elements; above, 40: 4096 x 8200 fp32 362, 4096 x 16384 629 (32 elements 383 and 516).
template <typename R, typename A, int VEC>
cudaError_t pick(NormParams& p, bool back, int rows_r, int rows_a, int sm, NormPlan* plan, cudaStream_t s) {
  const int n = span(p, VEC);
  if constexpr (VEC != kSkewed) {
    if (back) {
      if (n <= 8 * 512) return run<R, A, VEC, 8, 512, true>(p, rows_r, rows_a, sm, plan, s);
      if (n <= 16 * 512) return run<R, A, VEC, 16, 512, true>(p, rows_r, rows_a, sm, plan, s);
      return run<R, A, VEC, 40, 512, true>(p, rows_r, rows_a, sm, plan, s);
    }
  }
  if (n <= 8 * 32) return run<R, A, VEC, 8, 512, false, true>(p, rows_r, rows_a, sm, plan, s);
  if (n <= 8 * 992) return run<R, A, VEC, 8, 992, false>(p, rows_r, rows_a, sm, plan, s);
  return run<R, A, VEC, 24, 736, false>(p, rows_r, rows_a, sm, plan, s);
}

template <typename R, typename A>
cudaError_t pick_vec(NormParams& p, bool back, int vec, int rows_r, int rows_a, int sm,
                     NormPlan* plan, cudaStream_t s) {
  if (vec == kPieces) return pick<R, A, kPieces>(p, back, rows_r, rows_a, sm, plan, s);
  if (vec == kSkewed) return pick<R, A, kSkewed>(p, back, rows_r, rows_a, sm, plan, s);
  return pick<R, A, kOne>(p, back, rows_r, rows_a, sm, plan, s);
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

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s, NormPlan* plan_only) {
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
  const bool full = a.gate_kind == MOE_GATE_FULL, chan = a.gate_kind == MOE_GATE_CHANNEL;
  // every row of a token starts at the same place of a 16-byte (fp32: 32-byte) piece
  auto same = [&a](const void* q, long long ld) {
    return q == nullptr || ((reinterpret_cast<uintptr_t>(q) & 15u) == 0 && (ld - a.ld_residual) % 8 == 0);
  };
  const bool alike = same(a.residual, a.ld_residual) && same(a.branch, a.ld_branch) &&
                   same(a.out, a.ld_out) && same(a.h, a.ld_h) && same(a.d_out, a.ld_dout) &&
                   same(a.d_h, a.ld_dh) && (!full || (same(a.gate, a.ld_gate) && same(a.d_gate, a.ld_gate)));
  // pieces where every row starts at the same place of one (forward, 16384 x 7168:
  // 148 us, one column at a time 252); if that is not its start, the masks pay
  // forward only (16384 x 2001: 62 and 70; backward 8192 x 2001: 71 and 70, fp32
  // 81 and 73)
  const bool whole = a.H % 8 == 0 && a.ld_residual % 8 == 0;
  const int vec = !alike || (a.back && !whole) ? kOne : (whole ? kPieces : kSkewed);
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
  NormPlan own{};
  NormPlan* plan = plan_only != nullptr ? plan_only : &own;
  plan->only = plan_only != nullptr;
  cudaError_t e;
  if (a.residual_f32 && a.act_f32)
    e = pick_vec<float, float>(p, a.back, vec, rows_r, rows_a, sm, plan, s);
  else if (a.residual_f32)
    e = pick_vec<float, __nv_bfloat16>(p, a.back, vec, rows_r, rows_a, sm, plan, s);
  else
    e = pick_vec<__nv_bfloat16, __nv_bfloat16>(p, a.back, vec, rows_r, rows_a, sm, plan, s);
  if (e != cudaSuccess || p.n_part == 0 || plan->only) return e;
  const long long width = static_cast<long long>(p.n_part) * a.H;
  return launch_pdl(column_sum_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(32 * kSlices), 0,
                    s, static_cast<const float*>(a.part), plan->grid, p.n_part, a.H, o[0], o[1], o[2]);
}

}  // namespace moe
