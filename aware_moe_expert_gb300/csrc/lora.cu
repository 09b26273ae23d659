// A projection shared by all requests with a low-rank adapter per request:
//
//   y_t = x_t W^T + scale_a (x_t A_a^T) B_a^T,      a = adapter of token t (or none)
//
// and optionally SiLU(first half of y) * (second half).  x [T, K], W [N, K],
// A [n, r_max, K], B [n, N, r_max] bf16; rank_a <= r_max columns of an adapter
// count, what lies past them is not read into the result.
#include "gemm_common.cuh"
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

struct LoraParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  const int32_t* ranks;
  const float* scales;
  const int32_t* adapter;
  __nv_bfloat16* y;
  float* v;                // [T, r_max]
  long long ldx, ldy;
  int T, K, N, n, r_max, swiglu;
  int32_t* status;
};

// Adapter of token t, or -1; what is out of range is reported and is none.
__device__ __forceinline__ int adapter_of(const LoraParams& p, int t) {
  if (p.n == 0) return -1;
  const int a = __ldg(p.adapter + t);
  if (a < -1 || a >= p.n) {
    report(p.status, MOE_ERR_BAD_INDEX);
    return -1;
  }
  return a;
}
__device__ __forceinline__ int rank_of(const LoraParams& p, int a) {
  const int r = __ldg(p.ranks + a);
  if (r < 0 || r > p.r_max) {
    report(p.status, MOE_ERR_BAD_INDEX);
    return 0;
  }
  return r;
}

// v[t, i] = scale_a x_t . A_a[i]: a warp per token and rank.
__global__ void __launch_bounds__(256) lora_shrink_kernel(const LoraParams p) {
  pdl_wait_and_trigger();
  const long long id = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (id >= static_cast<long long>(p.T) * p.r_max) return;
  const int t = static_cast<int>(id / p.r_max), i = static_cast<int>(id - static_cast<long long>(t) * p.r_max);
  const int a = adapter_of(p, t);
  float v = 0.f;
  if (a >= 0 && i < rank_of(p, a)) {
    const uint4* xr = reinterpret_cast<const uint4*>(p.x + t * p.ldx);
    const uint4* ar = reinterpret_cast<const uint4*>(p.a + (static_cast<long long>(a) * p.r_max + i) * p.K);
    for (int q = lane; q < p.K / 8; q += 32) {
      const uint4 xv = __ldg(xr + q), av = __ldg(ar + q);
      const uint32_t* xs = &xv.x;
      const uint32_t* as = &av.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v = fmaf(bf16lo(xs[j]), bf16lo(as[j]), v);
        v = fmaf(bf16hi(xs[j]), bf16hi(as[j]), v);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    v *= __ldg(p.scales + a);
  }
  if (lane == 0) p.v[id] = v;
}

// 32 x 32 outputs a CTA, K in steps of 32 through shared memory.
__global__ void __launch_bounds__(256) lora_project_kernel(const LoraParams p) {
  __shared__ float xs[32][33], ws[2][32][33];
  pdl_wait_and_trigger();
  const int t0 = blockIdx.y * 32, n0 = blockIdx.x * 32;
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;   // column, first of four rows
  const int outs = p.swiglu ? p.N / 2 : p.N, parts = p.swiglu ? 2 : 1;
  float acc[2][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += 32) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r + 8 * i;
      const bool k_in = k0 + c < p.K;
      xs[row][c] = k_in && t0 + row < p.T ? __bfloat162float(p.x[(t0 + row) * p.ldx + k0 + c]) : 0.f;
      for (int h = 0; h < parts; ++h)
        ws[h][row][c] = k_in && n0 + row < outs
                            ? __bfloat162float(p.w[static_cast<long long>(h * outs + n0 + row) * p.K + k0 + c])
                            : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[0][i] = fmaf(xs[r + 8 * i][k], ws[0][c][k], acc[0][i]);
        if (p.swiglu) acc[1][i] = fmaf(xs[r + 8 * i][k], ws[1][c][k], acc[1][i]);
      }
  }
  if (n0 + c >= outs) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + r + 8 * i;
    if (t >= p.T) continue;
    const int a = adapter_of(p, t);
    if (a >= 0) {
      const int rank = rank_of(p, a);
      for (int h = 0; h < parts; ++h) {
        const __nv_bfloat16* br = p.b + (static_cast<long long>(a) * p.N + h * outs + n0 + c) * p.r_max;
        for (int j = 0; j < rank; ++j)
          acc[h][i] = fmaf(p.v[static_cast<long long>(t) * p.r_max + j], __bfloat162float(br[j]), acc[h][i]);
      }
    }
    const float o = p.swiglu ? silu_f(acc[0][i]) * acc[1][i] : acc[0][i];
    p.y[t * p.ldy + n0 + c] = __float2bfloat16_rn(o);
  }
}

}  // namespace

size_t lora_workspace_bytes(int T, int K, int N, int n, int r_max) {
  (void)K;
  (void)N;
  (void)n;
  return static_cast<size_t>(T) * r_max * 4;
}

cudaError_t launch_lora_project(const LoraArgs& g, cudaStream_t s) {
  LoraParams p{};
  p.x = static_cast<const __nv_bfloat16*>(g.x);
  p.w = static_cast<const __nv_bfloat16*>(g.w);
  p.a = static_cast<const __nv_bfloat16*>(g.a);
  p.b = static_cast<const __nv_bfloat16*>(g.b);
  p.ranks = g.ranks;
  p.scales = g.scales;
  p.adapter = g.adapter;
  p.y = static_cast<__nv_bfloat16*>(g.y);
  p.v = static_cast<float*>(g.ws);
  p.ldx = g.ldx;
  p.ldy = g.ldy;
  p.T = g.T;
  p.K = g.K;
  p.N = g.N;
  p.n = g.n_adapters;
  p.r_max = g.r_max;
  p.swiglu = g.swiglu;
  p.status = g.status;
  if (g.T == 0) return cudaSuccess;
  const long long warps = static_cast<long long>(g.T) * g.r_max;
  cudaError_t e = launch_pdl(lora_shrink_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)),
                             dim3(256), 0, s, p);
  if (e != cudaSuccess) return e;
  const int outs = g.swiglu ? g.N / 2 : g.N;
  return launch_pdl(lora_project_kernel, dim3((outs + 31) / 32, (g.T + 31) / 32), dim3(256), 0, s, p);
}

}  // namespace moe
