// Products of bf16 rows with packed 4-bit weights, dense or grouped by expert:
// y_r = x_r W^T, or with SwiGLU silu(x_r G^T) * (x_r U^T) of two matrices.
//
// The simplest form: a warp per output feature and eight rows, whole words of
// eight weights per lane, fp32 sums.
#include "gemm_common.cuh"
#include "moe_internal.h"
#include "quant.cuh"

namespace moe {
namespace {

constexpr int kRowsAtOnce = 8;
constexpr int kRowThreads = 256;

struct RowsParams {
  const __nv_bfloat16* x;
  const int32_t* token;
  const int32_t* offsets;
  const uint8_t* w;
  const float* factor;
  void* out;
  long long ldx, ldo, out_rows;
  size_t matrix;
  int dense_rows, x_rows, n, K, kb;
  int32_t* status;
};

template <int CODE, int GROUP, bool SWIGLU, bool F32>
__global__ void __launch_bounds__(kRowThreads) quant_rows_kernel(const RowsParams p) {
  pdl_wait_and_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.x * (kRowThreads / 32) + warp;
  const int g = blockIdx.y;
  const int first = p.offsets != nullptr ? p.offsets[g] : 0;
  const int last = p.offsets != nullptr ? p.offsets[g + 1] : p.dense_rows;
  if (first < 0 || last < first || last > p.out_rows) {
    if (threadIdx.x == 0) report(p.status, MOE_ERR_BAD_INDEX);
    return;
  }
  if (n >= p.n) return;
  constexpr int M = SWIGLU ? 2 : 1;
  constexpr uint32_t kRec = quant_record(GROUP);
  const uint8_t* rec0 = p.w + p.matrix * (static_cast<size_t>(g) * M) +
                        static_cast<size_t>(n / kQRows) * p.kb * kRec;
  const int r = n % kQRows;
  for (int t0 = first; t0 < last; t0 += kRowsAtOnce) {
    float acc[M][kRowsAtOnce] = {};
    const __nv_bfloat16* row[kRowsAtOnce];
    for (int i = 0; i < kRowsAtOnce; ++i) {
      int t = min(t0 + i, last - 1);
      if (p.token != nullptr) {
        t = p.token[t];
        if (t < 0 || t >= p.x_rows) {
          report(p.status, MOE_ERR_BAD_INDEX);
          t = 0;
        }
      }
      row[i] = p.x + t * p.ldx;
    }
    for (int v = lane; v < p.kb * 16; v += 32) {
      const int k = (v % 16) * 8, kk = v * 8;
      if (kk >= p.K) break;
      float w[M][8];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const uint8_t* rec = rec0 + p.matrix * m + static_cast<size_t>(v / 16) * kRec;
        uint32_t e[4];
        quant_expand<CODE>(
            *reinterpret_cast<const uint32_t*>(rec + quant_piece(r, (k % 32) / 8) + 4 * (k / 32)),
            QuantScale<CODE>(rec[kQCodeBytes + r * (kQK / GROUP) + k / GROUP]), e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[m][2 * i] = bf16lo(e[i]);
          w[m][2 * i + 1] = bf16hi(e[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kRowsAtOnce; ++i) {
        const uint4 q = *reinterpret_cast<const uint4*>(row[i] + kk);
        const uint32_t xv[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[m][i] = fmaf(w[m][2 * j], bf16lo(xv[j]), acc[m][i]);
            acc[m][i] = fmaf(w[m][2 * j + 1], bf16hi(xv[j]), acc[m][i]);
          }
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float f = p.factor[g * M + m] * quant_unit<CODE>();
#pragma unroll
      for (int i = 0; i < kRowsAtOnce; ++i) {
        for (int o = 16; o > 0; o >>= 1) acc[m][i] += __shfl_xor_sync(0xffffffffu, acc[m][i], o);
        acc[m][i] *= f;
      }
    }
    for (int i = 0; i < kRowsAtOnce; ++i) {
      if (lane != i || t0 + i >= last) continue;
      float y = 0.f;
#pragma unroll
      for (int j = 0; j < kRowsAtOnce; ++j)
        if (j == i) y = SWIGLU ? silu_f(acc[0][j]) * acc[M - 1][j] : acc[0][j];
      const size_t at = static_cast<size_t>(t0 + i) * p.ldo + n;
      if (F32)
        static_cast<float*>(p.out)[at] = y;
      else
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
    }
  }
}

template <int CODE, int GROUP>
cudaError_t launch_code(const QuantGemmArgs& a, const RowsParams& p, cudaStream_t s) {
  const dim3 grid((p.n + kRowThreads / 32 - 1) / (kRowThreads / 32), a.n_groups);
  if (a.swiglu)
    return launch_pdl(quant_rows_kernel<CODE, GROUP, true, false>, grid, dim3(kRowThreads), 0, s, p);
  return a.out_f32
             ? launch_pdl(quant_rows_kernel<CODE, GROUP, false, true>, grid, dim3(kRowThreads), 0, s, p)
             : launch_pdl(quant_rows_kernel<CODE, GROUP, false, false>, grid, dim3(kRowThreads), 0, s, p);
}

// out_t = sum_{j < k_t} w_{t,j} y[inv_row(t,j)] (+ y_shared[t]) of fp32 rows, in j
// order, rounded once.  A thread has four columns of a token.
__global__ void __launch_bounds__(128) combine_f32_kernel(
    const float4* __restrict__ y, const float4* __restrict__ y_shared,
    const int32_t* __restrict__ inv_row, const float* __restrict__ topk_w,
    const int32_t* __restrict__ kpt, int T, int nv, int k_max, int n_rows, uint2* __restrict__ out,
    int32_t* status) {
  pdl_wait_and_trigger();
  const long long gid = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int t = static_cast<int>(gid / nv), v = static_cast<int>(gid % nv);
  if (t >= T) return;
  const int k = min(max(kpt[t], 0), k_max);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  bool bad = false;
  for (int j0 = 0; j0 < k; j0 += 4) {
    float4 q[4];
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + i;
      const int r = j < k ? inv_row[static_cast<size_t>(t) * k_max + j] : -1;
      const bool ok = r >= 0 && r < n_rows;
      bad |= j < k && !ok;
      w[i] = ok ? topk_w[static_cast<size_t>(t) * k_max + j] : 0.f;
      q[i] = ok ? __ldcs(y + static_cast<size_t>(r) * nv + v) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc.x = fmaf(w[i], q[i].x, acc.x);
      acc.y = fmaf(w[i], q[i].y, acc.y);
      acc.z = fmaf(w[i], q[i].z, acc.z);
      acc.w = fmaf(w[i], q[i].w, acc.w);
    }
  }
  if (bad && v == 0) report(status, MOE_ERR_BAD_INDEX);
  if (y_shared != nullptr) {
    const float4 q = __ldcs(y_shared + static_cast<size_t>(t) * nv + v);
    acc.x += q.x;
    acc.y += q.y;
    acc.z += q.z;
    acc.w += q.w;
  }
  out[static_cast<size_t>(t) * nv + v] =
      make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

}  // namespace

cudaError_t launch_quant_gemm(const QuantGemmArgs& a, cudaStream_t s) {
  RowsParams p{};
  const QuantShape q = quant_shape(a.n, a.K, a.group);
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.token = a.token;
  p.offsets = a.offsets;
  p.w = static_cast<const uint8_t*>(a.w);
  p.factor = reinterpret_cast<const float*>(p.w + q.bytes * a.n_groups * (a.swiglu ? 2 : 1));
  p.out = a.out;
  p.ldx = a.ldx;
  p.ldo = a.ldo;
  p.out_rows = a.out_rows;
  p.matrix = q.bytes;
  p.dense_rows = a.dense_rows;
  p.x_rows = a.x_rows;
  p.n = a.n;
  p.K = a.K;
  p.kb = q.kb;
  p.status = a.status;
  if (a.code == MOE_QUANT_INT)
    return a.group == 16 ? launch_code<MOE_QUANT_INT, 16>(a, p, s)
                         : launch_code<MOE_QUANT_INT, 32>(a, p, s);
  return a.group == 16 ? launch_code<MOE_QUANT_E2M1, 16>(a, p, s)
                       : launch_code<MOE_QUANT_E2M1, 32>(a, p, s);
}

cudaError_t launch_combine_f32(const float* y, const float* y_shared, const int32_t* inv_row,
                               const float* topk_w, const int32_t* k_per_token, int T, int H,
                               int k_max, int n_rows, void* out, int32_t* status, cudaStream_t s) {
  const long long threads = static_cast<long long>(T) * (H / 4);
  return launch_pdl(combine_f32_kernel, dim3(static_cast<unsigned>((threads + 127) / 128)),
                    dim3(128), 0, s, reinterpret_cast<const float4*>(y),
                    reinterpret_cast<const float4*>(y_shared), inv_row, topk_w, k_per_token, T,
                    H / 4, k_max, n_rows, static_cast<uint2*>(out), status);
}

}  // namespace moe
