// Products of up to eight tokens with packed 4-bit weights: the projection, and the
// MoE layer's experts in two launches, without a permutation.
//
// A handful of tokens is bound by the weights' bytes and by latency, so the weights
// go from memory to registers to mma.m16n8k16 and nowhere else: a lane holds the
// 16-byte pieces of two rows (32 inputs each), which word by word are the A operands
// of two MMAs (quant.cuh); the tokens are the N side, all eight columns whatever
// their number, and a lane reads their inputs as they lie (16 bytes a word).  A warp
// multiplies 16 rows (or 16 gate and 16 up rows) by 128 inputs a step, kAhead steps
// in flight; the warps of a group split a task's steps and add their sums in shared
// memory in warp order, and where there are fewer tasks than CTAs, a cluster's CTAs
// split them further.
//
// Experts: every CTA lists the distinct units of the batch itself, from the router's
// selection.  The first launch computes act[t, j] = w_tj f_u silu(g) u of token t's
// j-th unit (its gate and its down matrix's factor with it, one rounding to bf16, as the bf16
// layer's activations have one; up to four tokens what it leaves is another bf16, in the
// columns that they leave free: the error of the outputs is then their own rounding's,
// 0.0016; from five tokens on there is no column for it, and the error 0.0023); the second
// one, whose weights stream while the first ends, multiplies 32 rows of W_down of ALL
// units and the shared expert with them, one long sum: the weighted sum over a token's
// units is part of it.
//
// Measured on a GB300: one token of K 7168, N 4096 5.7 us (2.9 TB/s); layers of 1, 8 and 3
// tokens (256 units of 384, k 16; the same; 256 of 2048 and a shared expert, k 8) 18.1, 41.0
// and 126 us; a shared expert alone (H 7168, 2048) of 1 and 8 tokens 12.4 and 14.2.  Loads of the codes alone, without products and tokens, take 3.8 us there, and
// 28 and 86 of the layers' 41.0 and 126: what is left is the expansion (issue slots 50-60%
// busy, ALU 40-54%), the tokens' loads, and for one token three launches' latencies.
#include <cfloat>
#include <type_traits>

#include "gemm_common.cuh"
#include "moe_internal.h"
#include "quant.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kTokens = kQuantFewTokens;
constexpr int kPairTokens = kQuantPairTokens;
static_assert(2 * kPairTokens == kTokens, "a second column for each");
constexpr int kMaxCluster = 8;

enum Mode { PROJECT, GATE_UP, DOWN };

// Steps in flight.  Three spill beside two tiles of rows (layer of eight tokens 41 us, 50) and
// gain nothing beside one (one token, K 7168, N 4096 5.7 us with both).
constexpr int kAhead = 2;
constexpr int kCtas = 2;
// Tiles of 16 rows of a task.  Two share the tokens' loads; a projection has few tasks
// and takes one (one token, K 7168, N 4096: 5.7 us, with two 6.5; eight tokens 7.1, 7.0).
__host__ __device__ constexpr int tiles_of(int mode, bool pair) { return mode == PROJECT && !pair ? 1 : 2; }

struct FewParams {
  const uint8_t* w;            // PROJECT, or the units' matrices
  const uint8_t* w_shared;
  const float* factor;         // of w's matrices
  const float* factor_shared;
  const float* factor_down;    // GATE_UP: of the matrices that the activations go to
  const float* factor_down_shared;
  const __nv_bfloat16* x;      // PROJECT, GATE_UP
  const __nv_bfloat16* act;    // DOWN: [T * k_max, I], act_shared [T, I_shared]
  const __nv_bfloat16* act_shared;
  const __nv_bfloat16* act_low;        // up to kPairTokens: what the roundings left
  const __nv_bfloat16* act_shared_low;
  __nv_bfloat16* out;          // PROJECT, DOWN
  __nv_bfloat16* out_act;      // GATE_UP
  __nv_bfloat16* out_act_shared;
  __nv_bfloat16* out_act_low;
  __nv_bfloat16* out_act_shared_low;
  const int32_t* topk_idx;     // [T, k_max]
  const float* topk_w;
  long long ldx, ldo;
  size_t matrix, matrix_shared;
  int T, n, K, kb;             // outputs of a matrix, its inputs, their records
  int n_shared, kb_shared, K_shared;   // GATE_UP: outputs; DOWN: inputs of the shared expert
  int E, k_max;
  int cluster;                 // CTAs that share a task
  int32_t* status;
};

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint4 ldg_nc(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two rows of a record as a lane holds them: a piece of each and its scales, in the low
// byte, or two.
struct Rows {
  uint4 c[2];
  uint32_t s[2];
};

// codes and scales: those of the lane's first row; its second one is eight rows on.
template <int GROUP>
__device__ __forceinline__ void load_rows(Rows& q, const uint8_t* codes, const uint8_t* scales) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    q.c[i] = ldg_stream(codes + i * 8 * 64);
    const uint8_t* at = scales + i * 8 * (kQK / GROUP);
    q.s[i] = GROUP == 32 ? __ldg(at) : __ldg(reinterpret_cast<const uint16_t*>(at));
  }
}

// d += rows x tokens over a record's 128 inputs; x: word w of the token's piece, four each.
template <int CODE, int GROUP>
__device__ __forceinline__ void multiply(float (&d)[4], const Rows& q, const uint4 (&x)[4]) {
  using Scale = QuantScale<CODE>;
  Scale sa[2], sb[2];          // of words 0 and 1, 2 and 3
  sa[0] = Scale::template at<0>(q.s[0]);
  sb[0] = Scale::template at<0>(q.s[1]);
  sa[1] = GROUP == 32 ? sa[0] : Scale::template at<1>(q.s[0]);
  sb[1] = GROUP == 32 ? sb[0] : Scale::template at<1>(q.s[1]);
  auto word = [&](auto index) {
    constexpr int W = decltype(index)::value;
    const uint32_t a = W == 0 ? q.c[0].x : W == 1 ? q.c[0].y : W == 2 ? q.c[0].z : q.c[0].w;
    const uint32_t b = W == 0 ? q.c[1].x : W == 1 ? q.c[1].y : W == 2 ? q.c[1].z : q.c[1].w;
    uint32_t ea[4], eb[4];
    quant_expand<CODE>(a, sa[W / 2], ea);
    quant_expand<CODE>(b, sb[W / 2], eb);
    mma_16816(d, ea[0], eb[0], ea[1], eb[1], x[W].x, x[W].y);
    mma_16816(d, ea[2], eb[2], ea[3], eb[3], x[W].z, x[W].w);
  };
  word(std::integral_constant<int, 0>());
  word(std::integral_constant<int, 1>());
  word(std::integral_constant<int, 2>());
  word(std::integral_constant<int, 3>());
}

// The batch's distinct units, ascending, and where each token has them.
struct Units {
  __align__(16) uint8_t slot[kMaxGroups][kTokens];   // j of token t's selection, 255: none
  uint8_t list[kMaxGroups];
  int warp_count[kWarps];
  int count;
};
static_assert(kMaxGroups == kWarps * 32, "a thread a unit");

__device__ __forceinline__ void list_units(Units& u, const FewParams& p, bool complain) {
  uint32_t* slots = reinterpret_cast<uint32_t*>(u.slot);
  for (int i = threadIdx.x; i < kMaxGroups * kTokens / 4; i += kWarps * 32) slots[i] = 0xFFFFFFFFu;
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * p.k_max; i += kWarps * 32) {
    const int t = i / p.k_max, e = p.topk_idx[i];
    if (e >= 0 && e < p.E) u.slot[e][t] = static_cast<uint8_t>(i - t * p.k_max);
    // a token without units gets the shared expert alone
    if (complain && e < 0 && i == t * p.k_max) report(p.status, MOE_ERR_K_RANGE);
  }
  __syncthreads();
  // thread = unit (256 of both)
  const uint2 s = *reinterpret_cast<const uint2*>(u.slot[threadIdx.x]);
  const bool used = (s.x & s.y) != 0xFFFFFFFFu;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t m = __ballot_sync(0xffffffffu, used);
  if (lane == 0) u.warp_count[warp] = __popc(m);
  __syncthreads();
  int at = __popc(m & ((1u << lane) - 1u));
  for (int w = 0; w < warp; ++w) at += u.warp_count[w];
  if (used) u.list[at] = static_cast<uint8_t>(threadIdx.x);
  if (threadIdx.x == 0) {
    int n = 0;
    for (int w = 0; w < kWarps; ++w) n += u.warp_count[w];
    u.count = n;
  }
  __syncthreads();
}

// Warps of a task: what makes the longest warp's steps fewest, with half a step for
// starting a task; the wider group on ties.
__device__ __forceinline__ int task_warps(int tasks, int steps, int ctas) {
  int best = kWarps;
  long long cost = 0x7fffffffffffll;
  for (int w = kWarps; w >= 1; w >>= 1) {
    const int at_once = ctas * (kWarps / w);
    const long long c = static_cast<long long>((tasks + at_once - 1) / at_once) * (2 * ((steps + w - 1) / w) + 1);
    if (c < cost) {
      cost = c;
      best = w;
    }
  }
  return best;
}

template <int MODE, int CODE, int GROUP, bool PAIR, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * 32, kCtas) quant_few_kernel(const FewParams p) {
  constexpr uint32_t kRec = quant_record(GROUP);
  constexpr int kTiles = tiles_of(MODE, PAIR);
  constexpr int kRows = PAIR ? 16 : 16 * kTiles;         // features of a task
  __shared__ Units units;
  __shared__ float sums[kWarps][kTiles * 16 * kTokens];
  __shared__ float parts[CLUSTER ? kMaxCluster : 1][kTiles * 16 * kTokens];   // of the cluster's CTAs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tig = lane & 3;
  // DOWN: token and part of the activations in this lane's column
  const bool pairs = p.T <= kPairTokens, low = pairs && g >= kPairTokens;
  const int token = pairs ? g & (kPairTokens - 1) : g;
  bool waited = false;
  // The selection was written before the launch that a DOWN launch follows, so it may
  // list the units and fetch weights at once.
  if (MODE == GATE_UP) {
    pdl_wait_and_trigger();
    waited = true;
  }
  int D = 1;
  if (MODE != PROJECT) {
    list_units(units, p, MODE == GATE_UP && blockIdx.x == 0);
    D = units.count;
  }
  const int tiles = (p.n + kRows - 1) / kRows;  // of a matrix
  const int shared_tiles = MODE == GATE_UP ? (p.n_shared + kRows - 1) / kRows : 0;
  const int tasks = MODE == GATE_UP ? D * tiles + shared_tiles : tiles;
  const int steps = MODE == DOWN ? D * p.kb + p.kb_shared : p.kb;
  const int rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
  const int ways = CLUSTER ? kWarps : task_warps(tasks, steps, gridDim.x);
  const int group = warp / ways, part = warp - group * ways;
  const int groups = kWarps / ways, stride = CLUSTER ? ways * p.cluster : ways;
  if (CLUSTER) cluster_sync_all();              // the peers run: their shared memory may be written

  for (int t0 = (CLUSTER ? blockIdx.x / p.cluster : blockIdx.x) * groups; t0 < tasks;
       t0 += (CLUSTER ? gridDim.x / p.cluster : gridDim.x) * groups) {
    const int task = t0 + group;
    const bool some = task < tasks;
    const bool shared = MODE == GATE_UP && task >= D * tiles;
    const int d = MODE == GATE_UP && !shared ? task / tiles : 0;
    const int tile = shared ? task - D * tiles : MODE == GATE_UP ? task - d * tiles : task;
    const int unit = MODE == GATE_UP && !shared && some ? units.list[d] : 0;
    const int r = tile * kRows % kQRows + g, rt = tile * kRows / kQRows;
    const uint32_t codes = quant_piece(r, tig), scales = kQCodeBytes + r * (kQK / GROUP) + tig * (32 / GROUP);
    // the task's rows in the first record that this warp reads
    const int start = rank * ways + part;
    // from the first tile of 16 rows to the second one
    const size_t next = !PAIR ? 16 * 64 : shared ? p.matrix_shared : p.matrix;
    const size_t next_scale = !PAIR ? 16 * (kQK / GROUP) : next;
    const uint8_t* rec = (shared ? p.w_shared : p.w + p.matrix * (static_cast<size_t>(unit) * (PAIR ? 2 : 1))) +
                         (static_cast<size_t>(rt) * p.kb + start) * kRec;

    float acc[kTiles][4] = {};
    Rows rows[kAhead][kTiles];
    uint4 x[kAhead][4];
    // DOWN counts through the units' records, then the shared expert's: unit, record, left
    int ws = start, wd = 0, wk = start;          // the next weights to load
    int xs = start, xd = 0, xk = start;          // the next inputs
    auto settle = [&](int& sd, int& sk) {
      while (sd < D && sk >= p.kb) {
        sk -= p.kb;
        ++sd;
      }
    };
    if (MODE == DOWN) {
      settle(wd, wk);
      xd = wd;
      xk = wk;
    }
    auto load_w = [&](Rows (&q)[kTiles]) {
      if (!some || ws >= steps) return;
      const uint8_t* at = rec;
      if (MODE != DOWN) {
        rec += static_cast<size_t>(stride) * kRec;
      } else {
        at = wd < D ? p.w + p.matrix * units.list[wd] + (static_cast<size_t>(rt) * p.kb + wk) * kRec
                    : p.w_shared + (static_cast<size_t>(rt) * p.kb_shared + wk) * kRec;
        wk += stride;
        settle(wd, wk);
      }
      load_rows<GROUP>(q[0], at + codes, at + scales);
      if (kTiles == 2) load_rows<GROUP>(q[kTiles - 1], at + codes + next, at + scales + next_scale);
      ws += stride;
    };
    auto load_x = [&](uint4 (&v)[4]) {
      if (!some || xs >= steps) return;
      const __nv_bfloat16* src = nullptr;
      int K = p.K;
      if (MODE != DOWN) {
        if (g < p.T) src = p.x + g * p.ldx;
      } else if (xd < D) {
        const int e = units.list[xd];
        const int j = units.slot[e][token];
        if (j != 255) src = (low ? p.act_low : p.act) + (static_cast<size_t>(token) * p.k_max + j) * p.K;
      } else {
        K = p.K_shared;
        if (token < p.T) src = (low ? p.act_shared_low : p.act_shared) + static_cast<size_t>(token) * K;
      }
      const int k = xk * kQK + 32 * tig;
      const int left = src != nullptr ? K - k : 0;
      src += k;
#pragma unroll
      for (int w = 0; w < 4; ++w) v[w] = 8 * w < left ? ldg_nc(src + 8 * w) : make_uint4(0u, 0u, 0u, 0u);
      xk += stride;
      if (MODE == DOWN) settle(xd, xk);
      xs += stride;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_w(rows[i]);
    if (!waited) {
      pdl_wait_and_trigger();
      waited = true;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_x(x[i]);
    if (some)
      for (int s = start; s < steps; s += kAhead * stride) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (s + i * stride >= steps) break;
#pragma unroll
          for (int j = 0; j < kTiles; ++j) multiply<CODE, GROUP>(acc[j], rows[i][j], x[i]);
          load_w(rows[i]);
          load_x(x[i]);
        }
      }
    // the group's sums: [row][token]
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      float2* to = reinterpret_cast<float2*>(sums[warp]) + (16 * j + g) * 4 + tig;
      to[0] = make_float2(acc[j][0], acc[j][1]);
      to[8 * 4] = make_float2(acc[j][2], acc[j][3]);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(ways * 32) : "memory");
    if (CLUSTER) {       // this CTA's sums to the first one's slots
      for (int i = threadIdx.x; i < kTiles * 16 * kTokens; i += kWarps * 32) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += sums[w][i];
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&parts[rank][i]), 0u)), "f"(v)
                     : "memory");
      }
      cluster_sync_all();
    }
    // rows fastest: neighbouring threads store neighbouring features
    for (int i = part * 32 + lane; some && rank == 0 && i < kRows * kTokens; i += ways * 32) {
      const int f = i % kRows, t = i / kRows, feature = tile * kRows + f;
      float v = 0.f, lift = 0.f;
      for (int w = 0; w < (CLUSTER ? p.cluster : ways); ++w) {
        const float* from = CLUSTER ? parts[w] : sums[group * ways + w];
        v += from[f * kTokens + t];
        if (MODE == DOWN && pairs && t < kPairTokens) v += from[f * kTokens + t + kPairTokens];
        if (PAIR) lift += from[(16 + f % 16) * kTokens + t];
      }
      if (t >= p.T || feature >= (shared ? p.n_shared : p.n)) continue;
      constexpr float u = quant_unit<CODE>();
      if (MODE == DOWN) {      // the factors came with the activations
        p.out[t * p.ldo + feature] = __float2bfloat16_rn(v);
        continue;
      }
      const float* factor = shared ? p.factor_shared : p.factor + 2 * unit;
      v *= factor[0] * u;
      if (PAIR) v = v / (1.f + expf(-v)) * (lift * (factor[1] * u));
      if (MODE == PROJECT) {
        p.out[t * p.ldo + feature] = __float2bfloat16_rn(v);
      } else {
        const int j = shared ? 0 : units.slot[unit][t];
        if (j == 255) continue;
        const size_t row = shared ? t : static_cast<size_t>(t) * p.k_max + j;
        const size_t at = row * (shared ? p.n_shared : p.n) + feature;
        v *= shared ? p.factor_down_shared[0] * u : p.factor_down[unit] * u * p.topk_w[row];
        const __nv_bfloat16 high = __float2bfloat16_rn(v);
        (shared ? p.out_act_shared : p.out_act)[at] = high;
        if (pairs) {           // 0, not NaN, where the rounding left infinity
          const float left = v - __bfloat162float(high);
          (shared ? p.out_act_shared_low : p.out_act_low)[at] =
              __float2bfloat16_rn(fabsf(left) <= FLT_MAX ? left : 0.f);
        }
      }
    }
    // the next task's sums overwrite these
    if (CLUSTER)
      cluster_sync_all();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(ways * 32) : "memory");
  }
  if (!waited) pdl_wait_and_trigger();
}

template <int MODE, int CODE, int GROUP, bool PAIR>
cudaError_t launch_kind(const FewParams& p, int grid, cudaStream_t s) {
  const dim3 b(kWarps * 32);
  if (p.cluster == 1) return launch_pdl(quant_few_kernel<MODE, CODE, GROUP, PAIR, false>, dim3(grid), b, 0, s, p);
  if constexpr (MODE == GATE_UP) return cudaErrorInvalidValue;   // has tasks enough
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = b;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, quant_few_kernel<MODE, CODE, GROUP, PAIR, MODE != GATE_UP>, p);
}

// `tasks` of about `steps` records: the CTAs of a cluster that share a task are what
// makes the longest CTA's steps fewest, with three for starting a task and three more for
// the cluster's barriers (clusters of 1, 2, 4 and 8: layer of 3 tokens, 224 tasks of 400 records,
// 126, 128, 134 and 161 us; layers of 8 and 1 tokens, 64 tasks of 384 and 48 records, 64, 48, 41
// and 47, and 19.8, 17.9, 18.2 and 21.2).
template <int MODE, bool PAIR>
cudaError_t launch_few(FewParams p, int code, int group, int tasks, int steps, int sm_count, cudaStream_t s) {
  const int ctas = kCtas * sm_count;
  if (ctas < 1) return cudaErrorNoDevice;      // the device could not be asked
  p.cluster = 1;
  if (MODE != GATE_UP) {
    long long best = 0;
    for (int c = 1; c <= kMaxCluster; c *= 2) {
      const long long rounds = (static_cast<long long>(tasks) * c + ctas - 1) / ctas;
      const long long cost = rounds * ((steps + kWarps * c - 1) / (kWarps * c) + (c > 1 ? 6 : 3));
      if (c == 1 || cost < best) {
        best = cost;
        p.cluster = c;
      }
    }
  }
  const int most = ctas / p.cluster * p.cluster;
  const int grid = MODE != GATE_UP && tasks * p.cluster < most ? tasks * p.cluster : most;
  if (code == MOE_QUANT_INT)
    return group == 16 ? launch_kind<MODE, MOE_QUANT_INT, 16, PAIR>(p, grid, s)
                       : launch_kind<MODE, MOE_QUANT_INT, 32, PAIR>(p, grid, s);
  return group == 16 ? launch_kind<MODE, MOE_QUANT_E2M1, 16, PAIR>(p, grid, s)
                     : launch_kind<MODE, MOE_QUANT_E2M1, 32, PAIR>(p, grid, s);
}

}  // namespace

cudaError_t launch_quant_project_few(const QuantGemmArgs& a, cudaStream_t s) {
  const QuantShape q = quant_shape(a.n, a.K, a.group);
  FewParams p{};
  p.w = static_cast<const uint8_t*>(a.w);
  p.factor = reinterpret_cast<const float*>(p.w + q.bytes * (a.swiglu ? 2 : 1));
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.ldx = a.ldx;
  p.ldo = a.ldo;
  p.matrix = q.bytes;
  p.T = a.dense_rows;
  p.n = a.n;
  p.K = a.K;
  p.kb = q.kb;
  p.status = a.status;
  const int tiles = (a.n + 15) / 16;
  return a.swiglu ? launch_few<PROJECT, true>(p, a.code, a.group, tiles, q.kb, a.sm_count, s)
                  : launch_few<PROJECT, false>(p, a.code, a.group, tiles, q.kb, a.sm_count, s);
}

cudaError_t launch_quant_ffn_few(const QuantFewArgs& a, cudaStream_t s) {
  const QuantShape gu = quant_shape(a.I, a.H, a.group), dn = quant_shape(a.H, a.I, a.group);
  const QuantShape gus = quant_shape(a.I_shared, a.H, a.group), dns = quant_shape(a.H, a.I_shared, a.group);
  FewParams p{};
  p.w = static_cast<const uint8_t*>(a.gate_up);
  p.w_shared = static_cast<const uint8_t*>(a.shared_gate_up);
  p.factor = reinterpret_cast<const float*>(p.w + gu.bytes * 2 * a.E);
  const uint8_t* down = static_cast<const uint8_t*>(a.down);
  const uint8_t* shared_down = static_cast<const uint8_t*>(a.shared_down);
  p.factor_down = reinterpret_cast<const float*>(down + dn.bytes * a.E);
  if (a.I_shared > 0) {
    p.factor_shared = reinterpret_cast<const float*>(p.w_shared + gus.bytes * 2);
    p.factor_down_shared = reinterpret_cast<const float*>(shared_down + dns.bytes);
  }
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.out_act = static_cast<__nv_bfloat16*>(a.act);
  p.out_act_shared = static_cast<__nv_bfloat16*>(a.act_shared);
  p.out_act_low = static_cast<__nv_bfloat16*>(a.act_low);
  p.out_act_shared_low = static_cast<__nv_bfloat16*>(a.act_shared_low);
  p.topk_idx = a.topk_idx;
  p.topk_w = a.topk_w;
  p.ldx = a.H;
  p.matrix = gu.bytes;
  p.matrix_shared = gus.bytes;
  p.T = a.T;
  p.n = a.I;
  p.K = a.H;
  p.kb = gu.kb;
  p.n_shared = a.I_shared;
  p.E = a.E;
  p.k_max = a.k_max;
  p.status = a.status;
  const cudaError_t e = launch_few<GATE_UP, true>(p, a.code, a.group, 0, 0, a.sm_count, s);
  if (e != cudaSuccess) return e;
  FewParams d = p;
  d.w = down;
  d.w_shared = shared_down;
  d.act = p.out_act;
  d.act_shared = p.out_act_shared;
  d.act_low = p.out_act_low;
  d.act_shared_low = p.out_act_shared_low;
  d.out = static_cast<__nv_bfloat16*>(a.out);
  d.ldo = a.H;
  d.matrix = dn.bytes;
  d.n = a.H;
  d.K = a.I;
  d.kb = dn.kb;
  d.n_shared = 0;
  d.K_shared = a.I_shared;
  d.kb_shared = a.I_shared > 0 ? dns.kb : 0;
  const int units = a.E < a.T * a.k_max ? a.E : a.T * a.k_max;       // at most
  return launch_few<DOWN, false>(d, a.code, a.group, (a.H + 31) / 32, units * dn.kb + d.kb_shared, a.sm_count, s);
}

}  // namespace moe
