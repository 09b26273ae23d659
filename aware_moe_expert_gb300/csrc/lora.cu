// A projection shared by all requests with a low-rank adapter per request:
//
//   y_t = x_t W^T + v_t B_a^T,   v_t = scale_a x_t A_a^T,   a = adapter of token t (or none)
//
// and optionally SiLU(first half of y) * (second half).  x [T, K], W [N, K],
// A [n, r_max, K], B [n, N, r_max] bf16, fp32 sums; of an adapter rank_a <= r_max
// rows of A and columns of B count.
//
// The adapters extend the reduction axis.  Of a tile of tokens, the distinct
// adapters' columns of B, in groups of 16, follow the K columns of W:
//
//   y[t, :] = [x_t | v_t placed in its adapter's columns, 0 elsewhere] [W | B_a0 | B_a1 ...]^T
//
// so a tile's adapters cost ceil(sum of their ranks / 64) more k-blocks of the
// same MMA loop, whatever the tokens' order, and no token is sorted or copied.
// The zeros only hide what is finite: a factor that is Inf or NaN counts as 0
// for everyone and is reported, so one request's adapter cannot reach another.
//
// v is rounded to bf16 once, being an MMA operand: 2^-9 of the adapter's term,
// below the rounding of y unless that term outgrows y.
#include <cudaTypedefs.h>

#include "gemm_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kRows = 128;              // M of one CTA's MMA
constexpr int kBK = 64;
constexpr int kGroup = 16;              // rank columns of a group: one MMA k-step
constexpr uint32_t kTile = kRows * kBK * 2;
constexpr int kWorkers = 128;           // threads that fill adapter k-blocks
constexpr int kMaxTileTokens = 256;

struct LoraParams {
  const __nv_bfloat16* b;
  const int32_t* ranks;
  const float* scales;
  const int32_t* adapter;
  __nv_bfloat16* v;                     // [T, r_max]
  __nv_bfloat16* y;
  long long ldy;
  int T, K, N, outs, n, r_max, swiglu;
  int wait_first;                       // no kernel of this call runs before this one
  int vec_y;                            // swap: 8-byte stores; pair: TMA stores
  int32_t* status;
};

// A group: adapter | first rank / 16 << 16 | columns in use (1..16) << 20.
__device__ __forceinline__ int grp_adapter(uint32_t g) { return static_cast<int>(g & 0xffffu); }
__device__ __forceinline__ int grp_first(uint32_t g) { return static_cast<int>((g >> 16) & 15u) * kGroup; }
__device__ __forceinline__ int grp_cols(uint32_t g) { return static_cast<int>(g >> 20); }

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

__device__ __forceinline__ void workers_sync() {
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

// Built by the 128 workers (e = 0..127): s_ad[n] the tokens' adapters, s_grp
// the groups of the distinct adapters in the order of their first token.
// Returns the number of groups.  s_sum: four words.
template <int NT>
__device__ __forceinline__ int build_groups(const LoraParams& p, int t0, int e, int* s_ad,
                                            uint32_t* s_grp, int* s_sum) {
  constexpr int PER = NT > kWorkers ? NT / kWorkers : 1;
  const int lane = e & 31, warp = e >> 5;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int n = e * PER + i;
    if (n < NT) s_ad[n] = t0 + n < p.T ? adapter_of(p, t0 + n) : -1;
  }
  workers_sync();
  int rank[PER], mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int n = e * PER + i;
    rank[i] = 0;
    if (n < NT) {
      const int a = s_ad[n];
      bool first = a >= 0 && (n == 0 || s_ad[n - 1] != a);
      for (int m = 0; first && m + 1 < n; ++m) first = s_ad[m] != a;
      if (first) rank[i] = rank_of(p, a);
      mine += (rank[i] + kGroup - 1) / kGroup;
    }
  }
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) s_sum[warp] = incl;
  workers_sync();
  int at = incl - mine, total = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < warp) at += s_sum[w];
    total += s_sum[w];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    for (int j = 0; j * kGroup < rank[i]; ++j)
      s_grp[at++] = static_cast<uint32_t>(s_ad[e * PER + i]) | (static_cast<uint32_t>(j) << 16) |
                    (static_cast<uint32_t>(min(kGroup, rank[i] - j * kGroup)) << 20);
  workers_sync();
  return total;
}

// Eight bf16 of a factor: those past `cols` and those that are not finite are 0.
__device__ __forceinline__ uint4 clean8(uint4 q, int cols, bool& bad) {
  uint32_t* w = &q.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo = w[i] & 0xffffu, hi = w[i] >> 16;
    if (2 * i >= cols) lo = 0u;
    if (2 * i + 1 >= cols) hi = 0u;
    if ((lo & 0x7f80u) == 0x7f80u) {
      bad = true;
      lo = 0u;
    }
    if ((hi & 0x7f80u) == 0x7f80u) {
      bad = true;
      hi = 0u;
    }
    w[i] = lo | (hi << 16);
  }
  return q;
}

// One k-block of four groups [g0, g0 + 4) of adapter columns, in the 128-byte
// swizzle that the MMA descriptors expect: the factor rows (128 rows, row i of
// W's row map(i), or none if map(i) < 0) and the tokens' v (VROWS rows).
template <int VROWS, typename Map>
__device__ __forceinline__ void fill_block(const LoraParams& p, int e, uint8_t* s_b, uint8_t* s_v,
                                           const int* s_ad, const uint32_t* s_grp, int g0, int groups,
                                           int t0, Map map) {
  const int c = e & 7, r0 = e >> 3;                    // 16-byte chunk of a row, first row
  const int gi = g0 + (c >> 1), half = (c & 1) * 8;
  const bool live = gi < groups;
  const uint32_t g = live ? s_grp[gi] : 0u;
  const int a = live ? grp_adapter(g) : -2;
  const int col = grp_first(g) + half, cols = live ? grp_cols(g) - half : 0;
  bool bad = false;
  uint4 q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int wr = map(r0 + 16 * i);
    q[i] = make_uint4(0u, 0u, 0u, 0u);
    if (cols > 0 && wr >= 0)
      q[i] = __ldg(reinterpret_cast<const uint4*>(
          p.b + (static_cast<long long>(a) * p.N + wr) * p.r_max + col));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    *reinterpret_cast<uint4*>(s_b + r * 128 + ((c ^ (r & 7)) << 4)) = clean8(q[i], cols, bad);
  }
#pragma unroll 8
  for (int i = 0; i < VROWS / 16; ++i) {
    const int r = r0 + 16 * i;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (cols > 0 && s_ad[r] == a)
      w = __ldcg(reinterpret_cast<const uint4*>(p.v + static_cast<long long>(t0 + r) * p.r_max + col));
    *reinterpret_cast<uint4*>(s_v + r * 128 + ((c ^ (r & 7)) << 4)) = w;
  }
  if (bad) report(p.status, MOE_ERR_NONFINITE);
}

// ---------------------------------------------------------------- v, few tokens
// v[t, i] = scale_a x_t . A_a[i]: 128 threads a (token, rank), all loads of a
// thread's slice in flight.  Columns past the rank are 0; a token without an
// adapter is left out (nothing reads its v).
constexpr int kDotThreads = 128;

__global__ void __launch_bounds__(kDotThreads) lora_dot_kernel(const LoraParams p,
                                                               const __nv_bfloat16* __restrict__ x,
                                                               const __nv_bfloat16* __restrict__ fa,
                                                               long long ldx) {
  __shared__ float s_part[kDotThreads / 32];
  pdl_wait_and_trigger();
  const int i = blockIdx.x, t = blockIdx.y;
  const int a = adapter_of(p, t);
  if (a < 0) return;
  const int rank = rank_of(p, a);
  float v = 0.f;
  if (i < rank) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + t * ldx);
    const uint4* ar = reinterpret_cast<const uint4*>(fa + (static_cast<long long>(a) * p.r_max + i) * p.K);
    const int nv = p.K / 8;
    for (int q0 = threadIdx.x; q0 < nv; q0 += 8 * kDotThreads) {
      uint4 xv[8], av[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = q0 + j * kDotThreads;
        xv[j] = q < nv ? __ldg(xr + q) : make_uint4(0u, 0u, 0u, 0u);
        av[j] = q < nv ? __ldg(ar + q) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t* xs = &xv[j].x;
        const uint32_t* as = &av[j].x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v = fmaf(bf16lo(xs[k]), bf16lo(as[k]), v);
          v = fmaf(bf16hi(xs[k]), bf16hi(as[k]), v);
        }
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = (s_part[0] + s_part[1]) + (s_part[2] + s_part[3]);
    p.v[static_cast<long long>(t) * p.r_max + i] =
        __float2bfloat16_rn(i < rank ? v * __ldg(p.scales + a) : 0.f);
  }
}

// ---------------------------------------------------------------- swapped operands
// D[128 rows of W (or of the adapters' A), NT tokens]: the weight rows are the
// MMA's M, so few tokens waste no tensor work and the weights stream once per
// token tile.  K is split over the S CTAs of a cluster; each leaves its fp32
// partial tile in shared memory and sums a slice of the tokens over the
// cluster in rank order.
//   SHRINK   rows = eight groups of factor rows (a TMA box of 16 rows each);
//            the sums are scaled and go to v where the token has that adapter
//   else     rows = 128 rows of W (swiglu: 64 gate and their 64 up rows), then
//            the adapters' k-blocks, filled by warps 2-5
// Warps: 0 TMA, 1 MMA, 2-5 adapter blocks, sums and stores.
template <int NT>
struct SwapCfg {
  static constexpr uint32_t kStage = kTile + NT * 128;
  static constexpr int kStages = NT >= 256 ? 3 : (NT >= 128 ? 4 : (NT >= 64 ? 6 : 8));
  static constexpr uint32_t kOffSlot = kStages * kStage;          // one adapter k-block
  static constexpr uint32_t kPitch = 132;                         // floats per token of the tile
  static constexpr uint32_t kRing = kOffSlot + kStage;
  static constexpr uint32_t kPart = NT * kPitch * 4;              // reuses the ring
  static constexpr uint32_t kOffBar = kRing > kPart ? kRing : kPart;
  static constexpr uint32_t kOffMisc = kOffBar + (2 * kStages + 3) * 8;
  static constexpr uint32_t kOffAd = kOffMisc + 64;
  static constexpr uint32_t kOffGrp = kOffAd + NT * 4;
  static constexpr uint32_t kUsed = kOffGrp + NT * 8 * 4;         // r_max 128: 8 groups a token
  static constexpr uint32_t kSmem = kUsed + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t kTmem = NT < 32 ? 32 : NT;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void store4(__nv_bfloat16* dst, float4 v, int left, bool vec) {
  if (vec && left >= 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    return;
  }
  if (left > 0) dst[0] = __float2bfloat16_rn(v.x);
  if (left > 1) dst[1] = __float2bfloat16_rn(v.y);
  if (left > 2) dst[2] = __float2bfloat16_rn(v.z);
  if (left > 3) dst[3] = __float2bfloat16_rn(v.w);
}

template <int NT, bool SHRINK>
__global__ void __launch_bounds__(192, 1)
    lora_swap_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const LoraParams p) {
  using C = SwapCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  uint64_t* lfull = empty + C::kStages;    // an adapter block is in its slot (or there is none)
  uint64_t* lempty = lfull + 1;
  uint64_t* tfull = lfull + 2;             // the accumulator is complete
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* s_last = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  int* s_total = reinterpret_cast<int*>(smem + C::kOffMisc + 12);
  int* s_sum = reinterpret_cast<int*>(smem + C::kOffMisc + 16);
  int* s_ad = reinterpret_cast<int*>(smem + C::kOffAd);
  uint32_t* s_grp = reinterpret_cast<uint32_t*>(smem + C::kOffGrp);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = gridDim.x, rank = blockIdx.x;
  const int t0 = blockIdx.z * NT;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(lfull, 4);
    mbar_init(lempty, 1);
    mbar_init(tfull, 1);
    *s_abort = 0;
    *s_last = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, C::kTmem);
    tmem_relinquish();
  }
  // The kernel that computes v has itself waited for everything before it, so
  // without wait_first all but v is ready; v is waited for where it is read.
  if (SHRINK || p.wait_first) asm volatile("griddepcontrol.wait;" ::: "memory");
  int groups = 0;
  if (SHRINK && warp >= 2) {
    groups = build_groups<NT>(p, t0, threadIdx.x - 64, s_ad, s_grp, s_sum);
    if (threadIdx.x == 64) *s_total = groups;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now: a dependent on this SM must not take the TMEM that this CTA needs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *s_tmem;
  const int KB = (p.K + kBK - 1) / kBK;
  const int kb0 = static_cast<int>(static_cast<long long>(KB) * rank / S);
  const int kb1 = static_cast<int>(static_cast<long long>(KB) * (rank + 1) / S);
  // SHRINK: blocks of eight groups, gridDim.y apart
  const int passes_end = SHRINK ? (*s_total + 7) / 8 : static_cast<int>(blockIdx.y) + 1;
  int stage = 0;
  uint32_t phase = 0, pass_parity = 0;
  for (int blk = blockIdx.y; blk < passes_end; blk += gridDim.y) {
    const int ng = SHRINK ? min(8, *s_total - blk * 8) : 0;
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t bytes = (SHRINK ? static_cast<uint32_t>(ng) * kGroup * kBK * 2 : kTile) + NT * 128;
        bool ok = *s_abort == 0;
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * C::kStage;
          mbar_expect_tx(&full[stage], bytes);
          if (SHRINK) {
            for (int g = 0; g < ng; ++g) {
              const uint32_t gr = s_grp[blk * 8 + g];
              tma_load_2d(sa + g * kGroup * kBK * 2, &tmW, &full[stage], kb * kBK,
                          grp_adapter(gr) * p.r_max + grp_first(gr));
            }
          } else if (p.swiglu) {
            tma_load_2d(sa, &tmW, &full[stage], kb * kBK, blk * 64);
            tma_load_2d(sa + kTile / 2, &tmW, &full[stage], kb * kBK, p.outs + blk * 64);
          } else {
            tma_load_2d(sa, &tmW, &full[stage], kb * kBK, blk * kRows);
          }
          tma_load_2d(sa + kTile, &tmX, &full[stage], kb * kBK, t0);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) {
          fail(s_abort, p.status);
          // the copies issued into the other slots end before the CTA does
          for (int s = 0; s < C::kStages; ++s) mbar_wait(&full[s], s < stage ? phase : phase ^ 1u, nullptr);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_bf16_f32(kRows, NT);
        bool ok = *s_abort == 0;
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, s_abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = sdesc_sw128(smem_u32(smem + stage * C::kStage));
          const uint64_t bd = sdesc_sw128(smem_u32(smem + stage * C::kStage + kTile));
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            umma_bf16(tmem, ad + 2u * k, bd + 2u * k, idesc, (kb != kb0 || k != 0) ? 1u : 0u);
          umma_commit(&empty[stage]);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!SHRINK) {
          const uint64_t ad = sdesc_sw128(smem_u32(smem + C::kOffSlot));
          const uint64_t bd = sdesc_sw128(smem_u32(smem + C::kOffSlot + kTile));
          for (uint32_t lp = 0; ok; lp ^= 1u) {
            if (!mbar_wait(lfull, lp, s_abort)) {
              ok = false;
              break;
            }
            if (*s_last == 2) break;       // nothing in the slot, nothing to follow
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) umma_bf16(tmem, ad + 2u * k, bd + 2u * k, idesc, 1u);
            umma_commit(lempty);
          }
        }
        if (!ok) fail(s_abort, p.status);
        umma_commit(tfull);
        if (!ok) mbar_wait(tfull, pass_parity, nullptr);
      }
      __syncwarp();
    } else {
      const int e = threadIdx.x - 64;
      if (!SHRINK) {
        if (!p.wait_first) asm volatile("griddepcontrol.wait;" ::: "memory");
        groups = build_groups<NT>(p, t0, e, s_ad, s_grp, s_sum);
        const int blocks = (groups + 3) / 4, half = p.swiglu ? 64 : kRows;
        auto map = [&](int i) {
          const int o = i < half ? blk * half + i : blk * half + i - half;
          return o < p.outs ? (i < half ? o : p.outs + o) : -1;
        };
        uint32_t lp = 0;
        for (int j = rank;; j += S) {
          int ok = 1;
          if (lane == 0) ok = mbar_wait(lempty, lp ^ 1u, s_abort) ? 1 : 0;
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) {
            if (lane == 0) fail(s_abort, p.status);
            break;
          }
          const bool more = j < blocks;
          if (more) {
            fill_block<NT>(p, e, smem + C::kOffSlot, smem + C::kOffSlot + kTile, s_ad, s_grp, 4 * j,
                           groups, t0, map);
            fence_proxy_async_smem();
          } else if (e == 0) {
            *s_last = 2;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(lfull);
          lp ^= 1u;
          if (!more) break;
        }
      }
      int ok = 1;
      if (lane == 0) ok = mbar_wait(tfull, pass_parity, s_abort) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      tc_fence_after();
      if (ok) {
        const int q = warp & 3;
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
        for (int n0 = 0; n0 < NT; n0 += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + n0, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (n0 + i < NT) part[(n0 + i) * C::kPitch + q * 32 + lane] = __uint_as_float(v[i]);
        }
      } else if (lane == 0) {
        fail(s_abort, p.status);
      }
      tc_fence_before();
    }
    pass_parity ^= 1u;
    __syncwarp();
    cluster_sync_all();      // every CTA's partial tile is in its shared memory
    if (warp >= 2) {
      const int per = NT / S;
      const uint32_t base = smem_u32(smem) + static_cast<uint32_t>(lane * 16);
      for (int n = rank * per + warp - 2; n < (rank + 1) * per; n += 4) {
        const int t = t0 + n;
        if (t >= p.T) break;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < S; ++q) {
          const float4 w = ld_cluster_f4(
              mapa_shared(base + static_cast<uint32_t>(n) * C::kPitch * 4, static_cast<uint32_t>(q)));
          v.x += w.x;
          v.y += w.y;
          v.z += w.z;
          v.w += w.w;
        }
        if (SHRINK) {
          const int g = blk * 8 + lane / 4;        // four rows of one group a lane
          if (lane / 4 < ng) {
            const uint32_t gr = s_grp[g];
            const int i0 = (lane & 3) * 4, cols = grp_cols(gr);
            if (s_ad[n] == grp_adapter(gr) && grp_first(gr) + i0 < p.r_max) {
              const float sc = __ldg(p.scales + grp_adapter(gr));
              v.x = i0 < cols ? v.x * sc : 0.f;
              v.y = i0 + 1 < cols ? v.y * sc : 0.f;
              v.z = i0 + 2 < cols ? v.z * sc : 0.f;
              v.w = i0 + 3 < cols ? v.w * sc : 0.f;
              store4(p.v + static_cast<long long>(t) * p.r_max + grp_first(gr) + i0, v, 4, true);
            }
          }
        } else if (p.swiglu) {
          float4 u;
          u.x = __shfl_down_sync(0xffffffffu, v.x, 16);
          u.y = __shfl_down_sync(0xffffffffu, v.y, 16);
          u.z = __shfl_down_sync(0xffffffffu, v.z, 16);
          u.w = __shfl_down_sync(0xffffffffu, v.w, 16);
          v.x = silu_f(v.x) * u.x;
          v.y = silu_f(v.y) * u.y;
          v.z = silu_f(v.z) * u.z;
          v.w = silu_f(v.w) * u.w;
          const int o = blk * 64 + lane * 4;
          if (lane < 16) store4(p.y + t * p.ldy + o, v, p.outs - o, p.vec_y);
        } else {
          const int o = blk * kRows + lane * 4;
          store4(p.y + t * p.ldy + o, v, p.outs - o, p.vec_y);
        }
      }
    }
    fence_proxy_async_smem();   // the next pass's copies land where the sums were
    __syncwarp();
    cluster_sync_all();      // nobody reads this CTA's tile any more
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// ---------------------------------------------------------------- CTA pairs, many tokens
// 256 tokens x 256 rows of W a tile (tcgen05 cta_group::2: each CTA holds 128
// token rows and half of the weight rows), persistent, accumulators double
// buffered in TMEM so that a tile's stores run under the next tile's MMAs.
// Warps: 0 TMA, 1 MMA (leader), 2-5 stores, 6-9 adapter k-blocks.  The
// adapters' warps run ahead: a tile's first block is in its slot long before
// the tile's K columns are done.
constexpr int kPairN = 256;
constexpr int kPairStages = 5;
constexpr int kPairThreads = 192 + kWorkers;
constexpr uint32_t kPairTmem = 2 * kPairN;

struct PairCfg {
  static constexpr uint32_t kStage = 2 * kTile;                   // 128 token rows, 128 W rows
  static constexpr uint32_t kOffSlot = kPairStages * kStage;
  static constexpr uint32_t kOffOut = kOffSlot + kStage;
  static constexpr uint32_t kOffBar = kOffOut + 4 * kStageRowsBytes;
  static constexpr uint32_t kOffMisc = kOffBar + (2 * kPairStages + 7) * 8;
  static constexpr uint32_t kOffAd = kOffMisc + 64;
  static constexpr uint32_t kOffGrp = kOffAd + kMaxTileTokens * 4;
  static constexpr uint32_t kUsed = kOffGrp + kMaxTileTokens * 8 * 4;
  static constexpr uint32_t kSmem = kUsed + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = globaltimer();
  while (true) {
    for (int i = 0; i < 64; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
      if (ok) return true;
    }
    if (abort != nullptr && *abort) return false;
    if (globaltimer() - t0 > kWaitLimitNs) return false;
  }
}

__device__ __forceinline__ void arrive_release_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__global__ void __launch_bounds__(kPairThreads, 1)
    lora_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmY, const LoraParams p) {
  using C = PairCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);   // leader
  uint64_t* empty = full + kPairStages;
  uint64_t* lfull = empty + kPairStages;   // leader: eight warps of the pair
  uint64_t* lempty = lfull + 1;
  uint64_t* tfull = lfull + 2;
  uint64_t* tempty = tfull + 2;            // leader
  uint64_t* done = tempty + 2;             // leader
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* s_more = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  int* s_sum = reinterpret_cast<int*>(smem + C::kOffMisc + 16);
  int* s_ad = reinterpret_cast<int*>(smem + C::kOffAd);
  uint32_t* s_grp = reinterpret_cast<uint32_t*>(smem + C::kOffGrp);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(lfull, 8);
    mbar_init(lempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8);
    }
    mbar_init(done, 1);
    *s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmY);
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, kPairTmem);
    tmem_relinquish_pair();
  }
  if (p.wait_first) asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *s_tmem;
  const int per_n = p.swiglu ? kPairN / 2 : kPairN;      // outputs of a tile
  const int n_tiles = (p.outs + per_n - 1) / per_n;
  const int total = (p.T + 255) / 256 * n_tiles;
  const int KB = (p.K + kBK - 1) / kBK;
  const int cid = static_cast<int>(blockIdx.x >> 1), ncl = static_cast<int>(gridDim.x >> 1);

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full_l = mapa_shared(smem_u32(full), 0);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int w = cid; ok && w < total; w += ncl) {
        const int mt = w / n_tiles, nt = w - mt * n_tiles;
        const int row = mt * 256 + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          const uint32_t fb = full_l + 8u * static_cast<uint32_t>(stage);
          uint8_t* sa = smem + stage * C::kStage;
          uint8_t* sb = sa + kTile;
          if (leader) mbar_expect_tx(&full[stage], 2 * C::kStage);
          tma_load_2d_pair(sa, &tmX, fb, kb * kBK, row);
          if (p.swiglu) {
            const int wr = nt * 128 + static_cast<int>(rank) * 64;
            tma_load_2d_pair(sb, &tmW, fb, kb * kBK, wr);
            tma_load_2d_pair(sb + kTile / 2, &tmW, fb, kb * kBK, p.outs + wr);
          } else {
            tma_load_2d_pair(sb, &tmW, fb, kb * kBK, nt * kPairN + static_cast<int>(rank) * 128);
          }
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) fail(s_abort, p.status);
      // every slot released: this CTA's loads have landed and no commit is
      // still aimed at its barriers
      for (int i = 0; ok && i < kPairStages; ++i) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, nullptr)) {
          fail(s_abort, p.status);
          break;
        }
        if (++stage == kPairStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader && lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(256, kPairN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, aphase = 0, lp = 0;
      bool ok = true;
      const uint64_t la = sdesc_sw128(smem_u32(smem + C::kOffSlot));
      const uint64_t lb = sdesc_sw128(smem_u32(smem + C::kOffSlot + kTile));
      for (int w = cid; ok && w < total; w += ncl) {
        if (!mbar_wait(&tempty[acc], aphase ^ 1u, s_abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * kPairN);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&full[stage], phase, s_abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = sdesc_sw128(smem_u32(smem + stage * C::kStage));
          const uint64_t bd = sdesc_sw128(smem_u32(smem + stage * C::kStage + kTile));
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            umma_bf16_pair(d, ad + 2u * k, bd + 2u * k, idesc, (kb | k) != 0 ? 1u : 0u);
          umma_commit_pair(&empty[stage], 0x3);
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        // the tile's adapter blocks; the slot that ends them holds none
        for (bool more = true; ok && more;) {
          if (!mbar_wait_cluster(lfull, lp, s_abort)) {
            ok = false;
            break;
          }
          more = *s_more != 0;
          if (more) {
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) umma_bf16_pair(d, la + 2u * k, lb + 2u * k, idesc, 1u);
          }
          umma_commit_pair(lempty, 0x3);
          lp ^= 1u;
        }
        if (!ok) break;
        umma_commit_pair(&tfull[acc], 0x3);
        if (++acc == 2) {
          acc = 0;
          aphase ^= 1u;
        }
      }
      if (!ok) fail(s_abort, p.status);
      umma_commit_pair(done, 0x1);
      mbar_wait(done, 0u, nullptr);
    }
    __syncwarp();
  } else if (warp < 6) {
    const int q = warp & 3;
    const uint32_t tempty_l = mapa_shared(smem_u32(tempty), 0);
    uint8_t* sbuf = smem + C::kOffOut + q * kStageRowsBytes;
    int acc = 0;
    uint32_t aphase = 0;
    for (int w = cid; w < total; w += ncl) {
      const int mt = w / n_tiles, nt = w - mt * n_tiles;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(&tfull[acc], aphase, s_abort) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0) fail(s_abort, p.status);
        break;
      }
      tc_fence_after();
      const uint32_t tbase =
          tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kPairN);
      const int row0 = mt * 256 + static_cast<int>(rank) * 128 + q * 32;
      const int t = row0 + lane;
#pragma unroll 1
      for (int ci = 0; ci < per_n / 32; ++ci) {
        uint32_t pk[16];
        if (p.swiglu) {
          // every 128 columns: gate(64) | up(64) of 64 outputs
          const int tc = (ci >> 1) * 128 + (ci & 1) * 32;
          uint32_t gv[32], uv[32];
          tmem_ld32(tbase + tc, gv);
          tmem_ld32(tbase + tc + 64, uv);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = pack_bf16x2(
                silu_f(__uint_as_float(gv[2 * i])) * __uint_as_float(uv[2 * i]),
                silu_f(__uint_as_float(gv[2 * i + 1])) * __uint_as_float(uv[2 * i + 1]));
        } else {
          uint32_t v[32];
          tmem_ld32(tbase + ci * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        }
        const int col = nt * per_n + ci * 32;
        if (p.vec_y) {
          if ((ci & 1) == 0) {
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          }
          stage_row_32(sbuf, lane, (ci & 1) * 4, pk);
          if ((ci & 1) != 0) {
            fence_proxy_async_smem();
            __syncwarp();
            // rows past T and columns past the outputs are clipped by the map
            if (lane == 0) {
              if (row0 < p.T && col - 32 < p.outs) tma_store_2d(&tmY, sbuf, col - 32, row0);
              bulk_commit();
            }
          }
        } else if (t < p.T) {
          __nv_bfloat16* dst = p.y + t * p.ldy + col;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (col + i < p.outs)
              dst[i] = __ushort_as_bfloat16(
                  static_cast<unsigned short>((i & 1) ? pk[i / 2] >> 16 : pk[i / 2] & 0xffffu));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_l + 8u * static_cast<uint32_t>(acc));
      if (++acc == 2) {
        acc = 0;
        aphase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  } else {
    const int e = threadIdx.x - 192;
    const uint32_t lfull_l = mapa_shared(smem_u32(lfull), 0);
    if (!p.wait_first) asm volatile("griddepcontrol.wait;" ::: "memory");
    uint32_t lp = 0;
    int built = -1, groups = 0;
    bool run = true;   // after a wait that gave up: keep the workers' barriers, touch nothing
    for (int w = cid; w < total; w += ncl) {
      const int mt = w / n_tiles, nt = w - mt * n_tiles;
      if (mt != built) {
        workers_sync();                    // the last tile's table is no longer read
        groups = build_groups<kMaxTileTokens>(p, mt * 256, e, s_ad, s_grp, s_sum);
        built = mt;
      }
      const int half = p.swiglu ? 64 : kRows;
      const int o0 = nt * per_n + static_cast<int>(rank) * half;
      auto map = [&](int i) {
        const int o = o0 + (i < half ? i : i - half);
        return o < p.outs ? (i < half ? o : p.outs + o) : -1;
      };
      const int blocks = (groups + 3) / 4;
      for (int j = 0; run && j <= blocks; ++j) {
        int ok = 1;
        if (lane == 0) ok = mbar_wait(lempty, lp ^ 1u, s_abort) ? 1 : 0;
        run = __shfl_sync(0xffffffffu, ok, 0) != 0;
        if (!run) {
          if (lane == 0) fail(s_abort, p.status);
          break;
        }
        if (j < blocks) {
          fill_block<kRows>(p, e, smem + C::kOffSlot + kTile, smem + C::kOffSlot,
                            s_ad + static_cast<int>(rank) * 128, s_grp, 4 * j, groups,
                            mt * 256 + static_cast<int>(rank) * 128, map);
          fence_proxy_async_smem();
        }
        if (e == 0) *s_more = j < blocks ? 1 : 0;
        __syncwarp();
        if (lane == 0) arrive_release_cluster(lfull_l);
        lp ^= 1u;
      }
    }
    // the last commit on this CTA's lempty has arrived
    if (run && lane == 0 && !mbar_wait(lempty, lp ^ 1u, nullptr)) fail(s_abort, p.status);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kPairTmem);
  }
}

// ---------------------------------------------------------------- host side

template <typename K, typename... Args>
cudaError_t launch_cluster(K kern, dim3 grid, int threads, int smem, int cluster, cudaStream_t s,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Tokens per tile of the swapped kernel.
int tile_tokens(int T) {
  if (T <= 16) return 16;
  if (T <= 32) return 32;
  if (T <= 64) return 64;
  if (T <= 128) return 128;
  return 256;
}

// From here up 256-token tiles of CTA pairs have enough tiles to fill the GPU.
constexpr int kPairMinT = 1025;
// Up to here (tokens x r_max) v is a dot product per (token, rank).
constexpr long long kDotMax = 2048;

template <int NT, bool SHRINK>
cudaError_t run_swap(const LoraArgs& g, const LoraParams& p, cudaStream_t s) {
  using C = SwapCfg<NT>;
  CUtensorMap tw, tx;
  if (SHRINK) {
    if (!encode_tmap_bf16(&tw, g.a, static_cast<long long>(g.n_adapters) * g.r_max, g.K, g.K, kGroup))
      return cudaErrorInvalidValue;
  } else if (!encode_tmap_bf16(&tw, g.w, g.N, g.K, g.K, g.swiglu ? 64 : kRows)) {
    return cudaErrorInvalidValue;
  }
  if (!encode_tmap_bf16(&tx, g.x, g.T, g.K, g.ldx, NT)) return cudaErrorInvalidValue;
  const int KB = (g.K + kBK - 1) / kBK;
  const int tt = (g.T + NT - 1) / NT;
  int rows;                               // blocks of 128 rows
  if (SHRINK) {
    const long long adapters = g.n_adapters < NT ? g.n_adapters : NT;
    const long long most = (adapters * ((g.r_max + kGroup - 1) / kGroup) + 7) / 8;
    const long long room = (2ll * g.sm_count + tt - 1) / tt;   // clusters walk over the rest
    rows = static_cast<int>(most < room ? most : room);
    if (rows < 1) rows = 1;
  } else {
    const int per = g.swiglu ? 64 : kRows;
    rows = (p.outs + per - 1) / per;
  }
  int S = 1;
  while (S < 8 && S * 2 <= KB && static_cast<long long>(rows) * tt * S * 2 <= g.sm_count) S *= 2;
  auto kern = lora_swap_kernel<NT, SHRINK>;
  static bool done[64] = {false};
  const cudaError_t e = set_smem_once(kern, static_cast<int>(C::kSmem), done);
  if (e != cudaSuccess) return e;
  return launch_cluster(kern, dim3(S, rows, tt), 192, static_cast<int>(C::kSmem), S, s, tw, tx, p);
}

template <bool SHRINK>
cudaError_t pick_swap(const LoraArgs& g, const LoraParams& p, cudaStream_t s) {
  switch (tile_tokens(g.T)) {
    case 16: return run_swap<16, SHRINK>(g, p, s);
    case 32: return run_swap<32, SHRINK>(g, p, s);
    case 64: return run_swap<64, SHRINK>(g, p, s);
    case 128: return run_swap<128, SHRINK>(g, p, s);
    default: return run_swap<256, SHRINK>(g, p, s);
  }
}

cudaError_t run_pair(const LoraArgs& g, const LoraParams& p, cudaStream_t s) {
  CUtensorMap tx, tw, ty;
  if (!encode_tmap_bf16(&tx, g.x, g.T, g.K, g.ldx, 128)) return cudaErrorInvalidValue;
  if (!encode_tmap_bf16(&tw, g.w, g.N, g.K, g.K, g.swiglu ? 64 : 128)) return cudaErrorInvalidValue;
  if (!p.vec_y)
    ty = tx;                              // not used
  else if (!encode_tmap_bf16(&ty, g.y, g.T, p.outs, g.ldy, 32))
    return cudaErrorInvalidValue;
  const int per_n = g.swiglu ? kPairN / 2 : kPairN;
  const long long tiles =
      static_cast<long long>((g.T + 255) / 256) * ((p.outs + per_n - 1) / per_n);
  if (tiles > (1ll << 30)) return cudaErrorInvalidValue;
  static bool done[64] = {false};
  cudaError_t e = set_smem_once(lora_pair_kernel, static_cast<int>(PairCfg::kSmem), done);
  if (e != cudaSuccess) return e;
  const int pairs = g.sm_count / 2 > 0 ? g.sm_count / 2 : 1;
  const int clusters = static_cast<int>(tiles < pairs ? tiles : pairs);
  return launch_cluster(lora_pair_kernel, dim3(2 * clusters), kPairThreads,
                        static_cast<int>(PairCfg::kSmem), 2, s, tx, tw, ty, p);
}

}  // namespace

size_t lora_workspace_bytes(int T, int r_max) { return static_cast<size_t>(T) * r_max * 2; }

cudaError_t launch_lora_project(const LoraArgs& g, cudaStream_t s) {
  LoraParams p{};
  p.b = static_cast<const __nv_bfloat16*>(g.b);
  p.ranks = g.ranks;
  p.scales = g.scales;
  p.adapter = g.adapter;
  p.v = static_cast<__nv_bfloat16*>(g.ws);
  p.y = static_cast<__nv_bfloat16*>(g.y);
  p.ldy = g.ldy;
  p.T = g.T;
  p.K = g.K;
  p.N = g.N;
  p.outs = g.swiglu ? g.N / 2 : g.N;
  p.n = g.n_adapters;
  p.r_max = g.r_max;
  p.swiglu = g.swiglu;
  p.status = g.status;
  p.wait_first = g.n_adapters == 0 ? 1 : 0;
  if (g.T == 0) return cudaSuccess;
  if (g.n_adapters > 0) {
    cudaError_t e;
    if (static_cast<long long>(g.T) * g.r_max <= kDotMax)
      e = launch_pdl(lora_dot_kernel, dim3(g.r_max, g.T), dim3(kDotThreads), 0, s, p,
                     static_cast<const __nv_bfloat16*>(g.x), static_cast<const __nv_bfloat16*>(g.a),
                     g.ldx);
    else
      e = pick_swap<true>(g, p, s);
    if (e != cudaSuccess) return e;
  }
  const uintptr_t y = reinterpret_cast<uintptr_t>(g.y);
  if (g.T >= kPairMinT) {
    p.vec_y = (y & 15u) == 0 && g.ldy % 8 == 0;
    return run_pair(g, p, s);
  }
  p.vec_y = (y & 7u) == 0 && g.ldy % 4 == 0;
  return pick_swap<false>(g, p, s);
}

}  // namespace moe
