// Packing of 4-bit weights (the layout is quant.cuh's): from a checkpoint's
// codes, scales and factors, from bf16 weights, and back to bf16.
//
// Set-up work, once a checkpoint.  A thread packs a scale group of a row: it loads codes a
// byte for each and sets a word's bits one by one; unpacking has a thread per word of
// eight weights.  Issue slots bound all three, not memory.  256 matrices of 768 x 2048, e2m1,
// groups of 16: packing 502 us (0.9 TB/s, issue slots 82% busy), quantising 1466 (the largest
// magnitudes 594, two bytes a lane at a time, 64 CTAs a matrix; then packing at 88%),
// unpacking 329 (3.1 TB/s, 81%).  One matrix of 4096 x 7168: 41, 864, where those 64 CTAs read
// it alone, and 25 us.
#include <cuda_fp8.h>

#include "moe_internal.h"
#include "quant.cuh"

namespace moe {
namespace {

constexpr int kPackThreads = 256;

// Waits for the launch before.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct PackParams {
  const uint8_t* codes;        // [count, rows, K / 2]; null: quantise w
  const uint8_t* scales;       // [count, rows, groups]
  const float* factors;        // [count]
  const __nv_bfloat16* w;      // [count, rows, K]
  __nv_bfloat16* w_out;        // unpack
  uint8_t* packed;
  int count, rows, K, code, group, groups;
  QuantShape shape;
  int32_t* status;
};

__device__ __forceinline__ float e4m3_value(uint32_t b) {
  const uint32_t e = (b >> 3) & 15u, m = b & 7u;
  return e != 0u ? ldexpf(1.f + 0.125f * m, static_cast<int>(e) - 7) : ldexpf(0.125f * m, -6);
}

// e4m3 bits without the sign as the stored byte; 0 for a scale of zero.
__device__ __forceinline__ uint32_t scale_byte(uint32_t b) {
  const uint32_t e = (b >> 3) & 15u, m = b & 7u;
  if (e != 0u) return (e + 9u) << 3 | m;
  if (m == 0u) return 0u;
  const int top = 31 - __clz(m);                 // m * 2^-9 = 2^(top - 9) * (m / 2^top)
  return static_cast<uint32_t>(top + 7) << 3 | ((m << (3 - top)) & 7u);
}

__device__ __forceinline__ uint32_t zero_code(int code) { return code == MOE_QUANT_INT ? 8u : 0u; }

// The code whose value is nearest to v (ties: the even code, as the formats round).
__device__ __forceinline__ uint32_t nearest(int code, float v) {
  if (code == MOE_QUANT_INT)
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(v), -8.f), 7.f)) + 8);
  const float a = fabsf(v);
  const uint32_t m = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) +
                     (a >= 3.5f) + (a > 5.f);
  return m | (signbit(v) ? 8u : 0u);
}

// Largest magnitude of each matrix, as ordered bits (all are >= 0).
__global__ void __launch_bounds__(kPackThreads) amax_kernel(PackParams p, uint32_t* amax) {
  pdl_wait();
  const size_t n = static_cast<size_t>(p.rows) * p.K;
  const __nv_bfloat16* w = p.w + n * blockIdx.y;
  float m = 0.f;
  bool bad = false;
  for (size_t i = static_cast<size_t>(blockIdx.x) * kPackThreads + threadIdx.x; i < n;
       i += static_cast<size_t>(gridDim.x) * kPackThreads) {
    const float v = fabsf(__bfloat162float(w[i]));
    if (v < INFINITY)
      m = fmaxf(m, v);
    else
      bad = true;
  }
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) atomicMax(amax + blockIdx.y, __float_as_uint(m));
  if (bad) report(p.status, MOE_ERR_NONFINITE);
}

__device__ __forceinline__ float vmax_of(int code) { return code == MOE_QUANT_INT ? 7.f : 6.f; }

// amax -> factor: the largest weight is the largest scale times the largest code.
__global__ void __launch_bounds__(kPackThreads) factor_kernel(PackParams p, float* factor) {
  pdl_wait();
  const int i = blockIdx.x * kPackThreads + threadIdx.x;
  if (i >= p.count) return;
  if (p.codes != nullptr) {
    const float f = p.factors[i];
    const bool bad = !(fabsf(f) < INFINITY);
    if (bad) report(p.status, MOE_ERR_NONFINITE);
    factor[i] = bad ? 0.f : f;                   // as a bad scale's weights
  } else {
    const float f = factor[i] / (448.f * vmax_of(p.code));
    factor[i] = f > 0.f ? f : 1.f;
  }
}

// Thread = one scale group of one row of one tile (its codes are 2 or 4 words),
// so that a scale is looked at once.
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackParams p,
                                                            const float* factor) {
  pdl_wait();
  const int per_row = kQK / p.group, words = p.group / 8;
  const size_t per_tile = static_cast<size_t>(kQRows) * per_row;
  const size_t per_matrix = per_tile * p.shape.rt * p.shape.kb;
  const size_t id = static_cast<size_t>(blockIdx.x) * kPackThreads + threadIdx.x;
  if (id >= per_matrix) return;
  for (int m = blockIdx.y; m < p.count; m += gridDim.y) {
    const size_t tile = id / per_tile;
    const int in = static_cast<int>(id - tile * per_tile);
    const int r = in / per_row, g = in - r * per_row;
    const int rt = static_cast<int>(tile / p.shape.kb), kb = static_cast<int>(tile % p.shape.kb);
    const int n = rt * kQRows + r, k0 = kb * kQK + g * p.group;
    uint8_t* rec = p.packed + p.shape.bytes * m + tile * quant_record(p.group);
    const bool real = n < p.rows && k0 < p.K;
    const size_t row = static_cast<size_t>(m) * p.rows + n;
    uint32_t sb = 0u;
    float step = 1.f;
    if (real && p.codes != nullptr) {
      const uint32_t b = p.scales[row * p.groups + k0 / p.group];
      // a scale is not negative, and not NaN (e4m3 has one, all exponent and mantissa bits)
      const bool bad = (b & 0x7Fu) == 0x7Fu || ((b & 0x80u) != 0u && (b & 0x7Fu) != 0u);
      if (bad) report(p.status, MOE_ERR_NONFINITE);
      sb = bad ? 0u : scale_byte(b & 0x7Fu);
    } else if (real) {
      float a = 0.f;
      const int end = min(k0 + p.group, p.K);
      for (int k = k0; k < end; ++k) {
        const float v = fabsf(__bfloat162float(p.w[row * p.K + k]));
        if (v < INFINITY) a = fmaxf(a, v);
      }
      const float want = a / (vmax_of(p.code) * factor[m]);
      const uint32_t b = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
      sb = scale_byte(b & 0x7Fu);
      step = e4m3_value(b & 0x7Fu) * factor[m];
    }
    rec[kQCodeBytes + r * per_row + g] = static_cast<uint8_t>(sb != 0u ? sb : 16u << 3);
    for (int j = 0; j < words; ++j) {
      const int k = g * p.group + 8 * j;         // within the tile
      uint32_t w = 0u;
      for (int i = 0; i < 8; ++i) {
        uint32_t q = zero_code(p.code);
        const int kk = kb * kQK + k + i;
        if (sb != 0u && kk < p.K) {
          if (p.codes != nullptr) {
            const uint32_t byte = p.codes[row * (p.K / 2) + kk / 2];
            q = (kk & 1) != 0 ? byte >> 4 : byte & 15u;
          } else {
            const float v = __bfloat162float(p.w[row * p.K + kk]);
            if (fabsf(v) < INFINITY) q = nearest(p.code, v / step);   // its reciprocal may be infinite
          }
        }
        w |= quant_place(p.code, q, i / 2, i & 1);
      }
      *reinterpret_cast<uint32_t*>(rec + quant_word(r, k / 32, (k % 32) / 8)) = w;
    }
  }
}

// Thread = one word: eight weights of a row.
template <int CODE>
__global__ void __launch_bounds__(kPackThreads) unpack_kernel(const PackParams p,
                                                              const float* factor) {
  pdl_wait();
  const int words = p.shape.kb * (kQK / 8);
  const size_t per_matrix = static_cast<size_t>(p.rows) * words;
  const size_t id = static_cast<size_t>(blockIdx.x) * kPackThreads + threadIdx.x;
  if (id >= per_matrix) return;
  const int n = static_cast<int>(id / words), v = static_cast<int>(id % words);
  const int kb = v / 16, k = (v % 16) * 8, r = n % kQRows;
  if (kb * kQK + k >= p.K) return;
  for (int m = blockIdx.y; m < p.count; m += gridDim.y) {
    const uint8_t* rec = p.packed + p.shape.bytes * m +
                         (static_cast<size_t>(n / kQRows) * p.shape.kb + kb) * quant_record(p.group);
    const uint32_t w =
        *reinterpret_cast<const uint32_t*>(rec + quant_word(r, k / 32, (k % 32) / 8));
    uint32_t e[4];
    quant_expand<CODE>(
        w, QuantScale<CODE>::template at<0>(rec[kQCodeBytes + r * (kQK / p.group) + k / p.group]), e);
    const float f = factor[m], u = quant_unit<CODE>();
    uint32_t o[4];
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(bf16lo(e[i]) * u * f, bf16hi(e[i]) * u * f);
    // K is a multiple of 8, so a word is whole or past the end
    *reinterpret_cast<uint4*>(p.w_out + (static_cast<size_t>(m) * p.rows + n) * p.K + kb * kQK + k) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Ends a packing.  Products read packed weights before they wait, and only a wait makes a
// launch's writes visible: that the packing does not trigger is not enough.  This thread waits
// for the packing, then triggers, so what starts behind it finds the weights complete.
__global__ void packed_kernel() { pdl_wait_and_trigger(); }

PackParams params_of(const QuantPackArgs& a) {
  PackParams p{};
  p.codes = static_cast<const uint8_t*>(a.codes);
  p.scales = static_cast<const uint8_t*>(a.scales);
  p.factors = a.factors;
  p.w = static_cast<const __nv_bfloat16*>(a.w);
  p.w_out = static_cast<__nv_bfloat16*>(a.w_out);
  p.packed = static_cast<uint8_t*>(a.packed);
  p.count = a.count;
  p.rows = a.rows;
  p.K = a.K;
  p.code = a.code;
  p.group = a.group;
  p.groups = (a.K + a.group - 1) / a.group;
  p.shape = quant_shape(a.rows, a.K, a.group);
  p.status = a.status;
  return p;
}

unsigned blocks(size_t n) { return static_cast<unsigned>((n + kPackThreads - 1) / kPackThreads); }

}  // namespace

size_t quant_bytes(int count, int rows, int K, int group) {
  return quant_shape(rows, K, group).bytes * count + static_cast<size_t>(count) * 4;
}

cudaError_t launch_quant_pack(const QuantPackArgs& a, cudaStream_t s) {
  const PackParams p = params_of(a);
  float* factor = reinterpret_cast<float*>(p.packed + p.shape.bytes * p.count);
  cudaError_t e;
  if (p.codes == nullptr) {
    e = cudaMemsetAsync(factor, 0, static_cast<size_t>(p.count) * 4, s);
    if (e != cudaSuccess) return e;
    const size_t n = static_cast<size_t>(p.rows) * p.K;
    for (int m0 = 0; m0 < p.count; m0 += 65535) {
      PackParams q = p;
      q.w += n * m0;
      const int m = p.count - m0 < 65535 ? p.count - m0 : 65535;
      const unsigned g = blocks(n) < 64u ? blocks(n) : 64u;
      e = launch_pdl(amax_kernel, dim3(g, m), dim3(kPackThreads), 0, s, q,
                     reinterpret_cast<uint32_t*>(factor) + m0);
      if (e != cudaSuccess) return e;
    }
  }
  e = launch_pdl(factor_kernel, dim3(blocks(p.count)), dim3(kPackThreads), 0, s, p, factor);
  if (e != cudaSuccess) return e;
  const size_t n = static_cast<size_t>(p.shape.rt) * p.shape.kb * kQRows * (kQK / p.group);
  e = launch_pdl(pack_kernel, dim3(blocks(n), p.count < 65535 ? p.count : 65535),
                 dim3(kPackThreads), 0, s, p, static_cast<const float*>(factor));
  return e != cudaSuccess ? e : launch_pdl(packed_kernel, dim3(1), dim3(1), 0, s);
}

cudaError_t launch_quant_unpack(const QuantPackArgs& a, cudaStream_t s) {
  const PackParams p = params_of(a);
  const float* factor = reinterpret_cast<const float*>(p.packed + p.shape.bytes * p.count);
  const size_t n = static_cast<size_t>(p.rows) * p.shape.kb * (kQK / 8);
  const dim3 grid(blocks(n), p.count < 65535 ? p.count : 65535);
  return a.code == MOE_QUANT_INT
             ? launch_pdl(unpack_kernel<MOE_QUANT_INT>, grid, dim3(kPackThreads), 0, s, p, factor)
             : launch_pdl(unpack_kernel<MOE_QUANT_E2M1>, grid, dim3(kPackThreads), 0, s, p, factor);
}

}  // namespace moe
