// A projection shared by all requests with a low-rank adapter per request:
//
//   y_t = x_t W^T + v_t B_a^T,   v_t = scale_a x_t A_a^T,   a = adapter of token t (or none)
//
// and optionally SiLU(first half of y) * (second half).  x [T, K], W [N, K],
// A [n, r_max, K], B [n, N, r_max] bf16, fp32 sums; of an adapter rank_a <= r_max
// rows of A and columns of B count.
//
// First a launch computes v, then one the projection; programmatic dependent
// launch lets the projection stream W meanwhile and meet v at its end.  There
// the adapters extend the reduction axis: of a tile of tokens, the distinct
// adapters' columns of B, in groups of 16, follow the K columns of W,
//   y[t, :] = [x_t | v_t in its adapter's columns, 0 elsewhere] [W | B_a0 | B_a1 ...]^T
// so a group costs two more k-steps of the same MMA loop (v is two operands),
// whatever the tokens' order; no token is sorted or copied.
//   few tokens   lora_swap_kernel: W's rows are the MMA's M, the weight stream
//                is the bound
//   many tokens  lora_pair_kernel: CTA pairs, the tensor cores are the bound
// v is kept in fp32; as an MMA operand it is two bf16, v = hi + lo, which take
// the adapter's k-steps twice (one bf16 of v put up to 2^-8 of the adapter's
// term into y, beside its own rounding, and y lost up to a third of its accuracy).
// The zeros only hide what is finite.  So that no token's result depends on
// another's adapter, a factor that is Inf or NaN counts as 0 and is reported:
// the pair kernel's warps look at the factors as they place them; the swapped
// kernel, which lets the TMA place them, keeps the adapters' sums apart and
// computes a tile's again with looked-over factors if one is not finite.
#include <algorithm>
#include <atomic>
#include <cmath>

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

struct LoraParams {   // what the kernels share
  const __nv_bfloat16* b;
  const int32_t* ranks;
  const float* scales;
  const int32_t* adapter;
  float* v;                             // [T, r_max]
  __nv_bfloat16* y;
  long long ldy;
  int T, K, N, outs, n, r_max, swiglu;
  int wait_first;                       // no kernel of this call runs before this one
  int vec_y;                            // pair: bytes of a store y is aligned for: 16 (TMA), 4 or 2
  int32_t* status;
};

// A group: adapter | first rank / 16 << 16 | columns in use (1..16) << 20.
__device__ __forceinline__ int grp_adapter(uint32_t g) { return static_cast<int>(g & 0xffffu); }
__device__ __forceinline__ int grp_first(uint32_t g) { return static_cast<int>((g >> 16) & 15u) * kGroup; }
__device__ __forceinline__ int grp_cols(uint32_t g) { return static_cast<int>(g >> 20); }

__device__ __forceinline__ int adapter_of(const LoraParams& p, int t) {
  if (p.n == 0) return -1;
  const int a = __ldcg(p.adapter + t);
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
// Returns the number of groups.  A hash table of the tile's adapters (4 NT
// keys and their first tokens, in s_grp's space, 8 NT words) finds the first
// tokens in a probe or two each; comparing every token with those before it
// took several us at 256 tokens.  s_sum: four words.
template <int NT>
__device__ __forceinline__ int build_groups(const LoraParams& p, int t0, int e, int* s_ad,
                                            uint32_t* s_grp, int* s_sum) {
  constexpr int PER = NT > kWorkers ? NT / kWorkers : 1;
  constexpr unsigned kSlots = 4 * NT;
  const int lane = e & 31, warp = e >> 5;
  int* key = reinterpret_cast<int*>(s_grp);
  int* first = key + kSlots;
  int ad[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int n = e * PER + i;
    ad[i] = n < NT && t0 + n < p.T ? adapter_of(p, t0 + n) : -1;
    if (n < NT) s_ad[n] = ad[i];
  }
  int rank[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) rank[i] = ad[i] >= 0 ? rank_of(p, ad[i]) : 0;
  for (int i = e; i < static_cast<int>(kSlots); i += kWorkers) {
    key[i] = -1;
    first[i] = NT;
  }
  workers_sync();
  unsigned at[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    at[i] = (static_cast<unsigned>(ad[i]) * 2654435761u >> 16) & (kSlots - 1);
    if (ad[i] >= 0) {
      for (;;) {      // ends: at most NT distinct keys in 4 NT slots
        const int was = atomicCAS(&key[at[i]], -1, ad[i]);
        if (was == -1 || was == ad[i]) break;
        at[i] = (at[i] + 1) & (kSlots - 1);
      }
      atomicMin(&first[at[i]], e * PER + i);
    }
  }
  workers_sync();
  int mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (ad[i] >= 0 && first[at[i]] != e * PER + i) rank[i] = 0;
    mine += (rank[i] + kGroup - 1) / kGroup;
  }
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) s_sum[warp] = incl;
  workers_sync();     // everyone is done with the hash table, too
  int to = incl - mine, total = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < warp) to += s_sum[w];
    total += s_sum[w];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    for (int j = 0; j * kGroup < rank[i]; ++j)
      s_grp[to++] = static_cast<uint32_t>(ad[i]) | (static_cast<uint32_t>(j) << 16) |
                    (static_cast<uint32_t>(min(kGroup, rank[i] - j * kGroup)) << 20);
  workers_sync();
  return total;
}

// Eight bf16 of a factor: those past `cols` and those that are not finite are 0.
__device__ __forceinline__ uint4 clean8(uint4 q, int cols, bool& bad) {
  uint32_t* w = &q.x;
  // an exponent of all ones carries into its half's top bit
  uint32_t carry = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) carry |= (w[i] & 0x7f807f80u) + 0x00800080u;
  if (cols >= 8 && (carry & 0x80008000u) == 0u) return q;
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

// Eight fp32 as two bf16 each: v = hi + lo to 2^-17 of v.
__device__ __forceinline__ void split8(const float4& a, const float4& b, uint4& hi, uint4& lo) {
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t* h = &hi.x;
  uint32_t* l = &lo.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    const float d0 = v[2 * i] - bf16lo(h[i]), d1 = v[2 * i + 1] - bf16hi(h[i]);
    // Inf and NaN are in hi
    l[i] = pack_bf16x2(fabsf(d0) < INFINITY ? d0 : 0.f, fabsf(d1) < INFINITY ? d1 : 0.f);
  }
}

// A worker's part of one k-block of four groups [4 j, 4 j + 4) of adapter
// columns: the 16-byte chunk c of every sixteenth factor row and token row, in
// the 128-byte swizzle that the MMA descriptors expect.
template <int VROWS>
struct Block {
  static constexpr int kV = VROWS / 16;
  uint4 b[8];
  int a, col, cols;

  // the chunk's place among the groups
  __device__ __forceinline__ void place(int e, const uint32_t* s_grp, int j, int groups) {
    const int gi = 4 * j + ((e & 7) >> 1), half = (e & 1) * 8;
    const bool live = gi < groups;
    const uint32_t g = live ? s_grp[gi] : 0u;
    a = live ? grp_adapter(g) : -2;
    col = grp_first(g) + half;
    cols = live ? grp_cols(g) - half : 0;
  }
  // factor row i is row map(i) of W (none if negative)
  template <typename Map>
  __device__ __forceinline__ void load_b(const LoraParams& p, int e, const uint32_t* s_grp, int j,
                                         int groups, Map map) {
    const int r0 = e >> 3;
    place(e, s_grp, j, groups);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int wr = map(r0 + 16 * i);
      b[i] = make_uint4(0u, 0u, 0u, 0u);
      if (cols > 0 && wr >= 0)
        b[i] = __ldg(reinterpret_cast<const uint4*>(
            p.b + (static_cast<long long>(a) * p.N + wr) * p.r_max + col));
    }
  }
  __device__ __forceinline__ static uint32_t chunk(int e) {
    const int c = e & 7, r0 = e >> 3;
    return static_cast<uint32_t>(r0 * 128 + ((c ^ (r0 & 7)) << 4));
  }
  __device__ __forceinline__ void store_b(const LoraParams& p, int e, uint8_t* s_b) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint4*>(s_b + chunk(e) + i * 2048) = clean8(b[i], cols, bad);
    if (bad) report(p.status, MOE_ERR_NONFINITE);
  }
  // token rows [16 i0, 16 i0 + 16 N) of the tile that begins at token t0
  template <int N>
  __device__ __forceinline__ void load_v(const LoraParams& p, int e, const int* s_ad, int t0, int i0,
                                         uint4 (&hi)[N], uint4 (&lo)[N]) {
    float4 x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = (e >> 3) + 16 * (i0 + i);
      x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (cols > 0 && s_ad[r] == a) {
        const float4* v =
            reinterpret_cast<const float4*>(p.v + static_cast<long long>(t0 + r) * p.r_max + col);
        x[i] = __ldcg(v);
        y[i] = __ldcg(v + 1);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) split8(x[i], y[i], hi[i], lo[i]);
  }
  template <int N>
  __device__ __forceinline__ static void store_v(int e, int i0, uint8_t* s_v, const uint4 (&w)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<uint4*>(s_v + chunk(e) + (i0 + i) * 2048) = w[i];
  }
  // the whole v tile, hi and behind it lo
  __device__ __forceinline__ void put_v(const LoraParams& p, int e, const int* s_ad, int t0, uint8_t* s_v) {
    constexpr int N = kV < 8 ? kV : 8;
#pragma unroll
    for (int i0 = 0; i0 < kV; i0 += N) {
      uint4 hi[N], lo[N];
      load_v<N>(p, e, s_ad, t0, i0, hi, lo);
      store_v<N>(e, i0, s_v, hi);
      store_v<N>(e, i0, s_v + VROWS * 128, lo);
    }
  }
};

// ---------------------------------------------------------------- v, few tokens
// v[t, i] = scale_a x_t . A_a[i]: a CTA for a token and eight ranks, x read once
// for the eight.  Columns past the rank are 0; a token without an adapter is
// left out (nothing reads its v).  The chain of dependent loads is two long:
// the adapter's index, then its rank, scale and rows together (rows past the
// rank exist in the pool and are not used).
// Bound: A's rows, read from L2 once per token: 1024 tokens, K 7168, r 16 in about
// 30 us, 9 TB/s; below 64 tokens the chain, 4-5 us.
constexpr int kDotThreads = 256;
constexpr int kDotRanks = 8;
constexpr int kDotVecs = 2;      // 16-byte vectors of a row a thread has in flight

__global__ void __launch_bounds__(kDotThreads, 2)
    lora_dot_kernel(const LoraParams p, const __nv_bfloat16* __restrict__ x,
                    const __nv_bfloat16* __restrict__ fa, long long ldx) {
  __shared__ float s_part[kDotThreads / 32][kDotRanks];
  pdl_wait_and_trigger();
  const int i0 = blockIdx.x * kDotRanks, t = blockIdx.y;
  const int nv = p.K / 8;
  const uint4* xr = reinterpret_cast<const uint4*>(x + t * ldx);
  const int a = adapter_of(p, t);
  if (a < 0) return;
  const float scale = __ldg(p.scales + a);
  const int rank = rank_of(p, a);
  const uint4* ar = reinterpret_cast<const uint4*>(fa + (static_cast<long long>(a) * p.r_max + i0) * p.K);
  float v[kDotRanks] = {};
  for (int q0 = threadIdx.x; q0 < nv; q0 += kDotVecs * kDotThreads) {
    uint4 xv[kDotVecs], av[kDotVecs][kDotRanks];
#pragma unroll
    for (int j = 0; j < kDotVecs; ++j) {
      const int q = q0 + j * kDotThreads;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      xv[j] = q < nv ? __ldg(xr + q) : zero;
#pragma unroll
      for (int i = 0; i < kDotRanks; ++i)
        av[j][i] = q < nv ? __ldg(ar + static_cast<long long>(i) * nv + q) : zero;
    }
#pragma unroll
    for (int j = 0; j < kDotVecs; ++j) {
      const uint32_t* xs = &xv[j].x;
#pragma unroll
      for (int i = 0; i < kDotRanks; ++i) {
        const uint32_t* as = &av[j][i].x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[i] = fmaf(bf16lo(xs[k]), bf16lo(as[k]), v[i]);
          v[i] = fmaf(bf16hi(xs[k]), bf16hi(as[k]), v[i]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kDotRanks; ++i)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < kDotRanks; ++i) s_part[threadIdx.x >> 5][i] = v[i];
  }
  __syncthreads();
  if (threadIdx.x < kDotRanks) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kDotThreads / 32; ++w) sum += s_part[w][threadIdx.x];
    const int i = i0 + threadIdx.x;
    p.v[static_cast<long long>(t) * p.r_max + i] = i < rank ? sum * scale : 0.f;
  }
}

// ---------------------------------------------------------------- swapped operands
// D[128 rows of W (or of the adapters' A), NT tokens]: the weight rows are the
// MMA's M, so few tokens waste no tensor work and the weights stream once per
// token tile.  K is split over the S CTAs of a cluster; rank q owns tokens
// [q NT/S, (q+1) NT/S) of the tile: every CTA pushes its fp32 partial sums of
// them into q's shared memory (stores need no round trip; reading them from
// the other CTAs took 6 us for 64 tokens of four), and q adds them in rank order.
//   SHRINK   rows = eight groups of factor rows (a TMA box of 16 rows each);
//            the sums are scaled and go to v where the token has that adapter
//   else     rows = 128 rows of W (swiglu: 64 gate and their 64 up rows)
// The adapters' k-blocks are dealt to the CTAs of the cluster and come through
// the same ring behind the K columns (factor rows in TMA boxes of 16 columns);
// their sums have columns of their own in TMEM.  How much of W is in flight is
// kept to what the bandwidth needs: with 16 MB of it, every other load waited
// 2-3 us, and v with its chain of loads came late.
// Warps: 0 TMA, 1 MMA, 2-5 v tiles, sums and stores: a thread has the row of
// its TMEM lane.
// Bound: W's stream.  K 7168, N 4096: one token 13.6 us without adapters (4.3 TB/s
// of W; the rest is the way to its first bytes and the exchange of the sums),
// 14.5 with one of rank 16, v's kernel under it; 64 tokens 15.4 without, 23.0 with
// 48 adapters of up to rank 32, whose v comes 4-5 us late and whose groups' slots
// take the rest.  SHRINK, K 7168, r 64, 1024 tokens: 92 us with an adapter each,
// 33 in requests of 64 (with a projection to 128 outputs behind it).
template <int NT, bool SHRINK>
struct SwapCfg {
  static constexpr uint32_t kStage = kTile + NT * 128;
  static constexpr int kStages = NT >= 256 ? (SHRINK ? 4 : 3) : (NT >= 128 ? (SHRINK ? 5 : 4) : 6);
  static constexpr int kG = NT <= 128 ? 4 : 2;                    // groups of adapter columns a v slot holds
  static constexpr int kVSlots = SHRINK ? 0 : (NT >= 64 ? 2 : 4);
  static constexpr uint32_t kVTile = NT * kGroup * 2;
  static constexpr uint32_t kVBytes = 2 * kG * kVTile;            // v of each group: hi, lo
  static constexpr uint32_t kOffV = kStages * kStage;
  static constexpr uint32_t kOffBar = kOffV + kVSlots * kVBytes;
  static constexpr uint32_t kOffMisc = kOffBar + (2 * kStages + 3 + 2 * kVSlots) * 8;
  static_assert(SHRINK || kVSlots * kVBytes >= 2 * NT * 128, "look_over has a whole block there");
  static constexpr uint32_t kOffAd = kOffMisc + 64;
  static constexpr uint32_t kOffGrp = kOffAd + NT * 4;
  static constexpr uint32_t kUsed = kOffGrp + NT * 8 * 4;
  static constexpr uint32_t kSmem = kUsed + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(NT * kRows * 4 <= kOffV, "the partial sums reuse the ring");
  static constexpr uint32_t kCols = NT < 32 ? 32 : NT;            // loads read 32 columns
  static constexpr uint32_t kTmem = SHRINK ? kCols : 2 * kCols;   // projection: the adapters' sums, too
};

// A worker's part of v of G groups for NT tokens: a chunk of eight columns of one
// of the groups, of every (64 / G)th token.
template <int NT, int G>
struct VRows {
  static constexpr int kStep = 64 / G, kN = NT < kStep ? 1 : NT / kStep;
  float4 v[kN][2];
  unsigned own;           // bit i: the i-th of them has this adapter

  __device__ __forceinline__ void load(const LoraParams& p, const int* s_ad, const uint32_t* s_grp,
                                       int gi, int groups, int t0, int e) {
    const int half = e & 1, r0 = e / (2 * G);
    gi += (e >> 1) % G;
    const uint32_t g = gi < groups ? s_grp[gi] : 0u;
    const bool live = gi < groups && grp_cols(g) > 8 * half;
    const int a = grp_adapter(g), col = grp_first(g) + 8 * half;
    own = 0u;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = r0 + kStep * i;
      if (live && r < NT && s_ad[r] == a) {
        own |= 1u << i;
        const float4* from =
            reinterpret_cast<const float4*>(p.v + static_cast<long long>(t0 + r) * p.r_max + col);
        v[i][0] = __ldcg(from);
        v[i][1] = __ldcg(from + 1);
      }
    }
  }
  // each group's tile of 16 columns in the 32-byte swizzle, hi and behind it lo
  __device__ __forceinline__ void store(uint8_t* to, int e) const {
    const int half = e & 1, r0 = e / (2 * G);
    to += (e >> 1) % G * (NT * kGroup * 4);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = r0 + kStep * i;
      if (r >= NT) break;
      uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
      if (own >> i & 1u) split8(v[i][0], v[i][1], hi, lo);
      uint8_t* at = to + r * 32 + ((half ^ ((r >> 2) & 1)) << 4);
      *reinterpret_cast<uint4*>(at) = hi;
      *reinterpret_cast<uint4*>(at + NT * kGroup * 2) = lo;
    }
  }
};

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Descriptor of a K-major tile of 16 bf16 columns (rows of 32 bytes, 32-byte
// swizzle, groups of eight rows 256 bytes apart), as a TMA load with
// CU_TENSOR_MAP_SWIZZLE_32B writes it.
__device__ __forceinline__ uint64_t sdesc_sw32(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(256 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(6) << 61;
  return d;
}

// SiLU within (4 + 1.2 |g|) 2^-23 of its value where g > -87 (the bounds of __expf and
// __fdividef; 2^-16 at the end, 2^-20 from -4 up), 0 where it is below 2^-119.  y is
// rounded to 2^-8 of its value (4392 tokens, K 808, 1472 outputs, one adapter: 40 us; exact
// division 66).
__device__ __forceinline__ float silu_fast(float g) { return __fdividef(g, 1.f + __expf(-g)); }

// SHRINK: what row `row` of a tile of eight groups is, a column of v of one
// adapter; the lanes of a warp have two groups.
struct ShrinkRow {
  int a, col, a0, a1;
  bool live, use;
  float scale;
  __device__ __forceinline__ ShrinkRow(const LoraParams& p, const uint32_t* grp, int ng, int row) {
    const int g = row / kGroup;
    const uint32_t gr = g < ng ? grp[g] : 0u;
    a = g < ng ? grp_adapter(gr) : -2;
    col = grp_first(gr) + row % kGroup;
    live = g < ng && col < p.r_max;
    use = row % kGroup < grp_cols(gr);  // past the rank v is 0
    scale = g < ng ? __ldg(p.scales + a) : 0.f;
    a0 = __shfl_sync(0xffffffffu, a, 0);
    a1 = __shfl_sync(0xffffffffu, a, 16);
  }
  // by the whole warp, `ad` the adapter of the lane's token: the tokens whose
  // adapter the calling lane's group belongs to
  __device__ __forceinline__ unsigned tokens(int ad) const {
    const unsigned m0 = __ballot_sync(0xffffffffu, ad == a0), m1 = __ballot_sync(0xffffffffu, ad == a1);
    return !live ? 0u : (a == a0 ? m0 : m1);
  }
  __device__ __forceinline__ void put(const LoraParams& p, int t, float v) const {
    p.v[static_cast<long long>(t) * p.r_max + col] = use ? v * scale : 0.f;
  }
};

// Sums the S partial rows of this CTA's tokens, in rank order, and stores them;
// a thread has row `row` of the tile.
template <bool SHRINK, int S>
__device__ __forceinline__ void finish(const LoraParams& p, const float* part, const int* ad,
                                       const uint32_t* grp, int ng, int first, int count, int per,
                                       int blk, int row) {
  auto sum = [&](int n, int r) {
    float w[S];
#pragma unroll
    for (int s = 0; s < S; ++s) w[s] = part[(s * per + n) * kRows + r];
    float v = w[0];
#pragma unroll
    for (int s = 1; s < S; ++s) v += w[s];
    return v;
  };
  if (SHRINK) {
    const ShrinkRow m(p, grp, ng, row);
    for (int n0 = 0; n0 < count; n0 += 32) {
      unsigned mine = m.tokens(n0 + (row & 31) < count ? ad[n0 + (row & 31)] : -1);
      while (mine != 0u) {              // up to four tokens' loads at a time
        int n[4];
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          n[k] = mine != 0u ? n0 + __ffs(mine) - 1 : -1;
          mine &= mine - 1u;
          v[k] = n[k] >= 0 ? sum(n[k], row) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n[k] >= 0) m.put(p, first + n[k], v[k]);
      }
    }
  } else if (p.swiglu) {
    const int o = blk * 64 + (row & 63);
    if (o >= p.outs) return;
    __nv_bfloat16* y = p.y + first * p.ldy + o;
#pragma unroll 4
    for (int n = row >> 6; n < count; n += 2)
      y[n * p.ldy] = __float2bfloat16_rn(silu_fast(sum(n, row & 63)) * sum(n, (row & 63) + 64));
  } else {
    const int o = blk * kRows + row;
    if (o >= p.outs) return;
    __nv_bfloat16* y = p.y + first * p.ldy + o;
#pragma unroll 8
    for (int n = 0; n < count; ++n) y[n * p.ldy] = __float2bfloat16_rn(sum(n, row));
  }
}

// Row i of a tile of W (swiglu: 64 gate rows, then their up rows) as a row of W,
// or -1.
__device__ __forceinline__ int tile_row(const LoraParams& p, int blk, int i) {
  const int half = p.swiglu ? 64 : kRows;
  const int o = blk * half + (i < half ? i : i - half);
  return o < p.outs ? (i < half ? o : p.outs + o) : -1;
}

// By the workers, once every MMA of the CTA is complete: if one of its
// adapters' sums is not finite, they are all computed again with factors that
// were looked over.  The same k-steps in the same order: what was finite keeps
// its bits.  The ring is free by then.
template <int NT>
__device__ __forceinline__ void look_over(const LoraParams& p, uint8_t* smem, const int* s_ad,
                                          const uint32_t* s_grp, int* s_sum, uint64_t* redo,
                                          volatile int* s_abort, uint32_t tmem, int blk, int t0,
                                          int rank, int S, int groups, int e) {
  using C = SwapCfg<NT, false>;
  const int warp = e >> 5, lane = e & 31, q = (warp + 2) & 3;
  tc_fence_after();
  bool bad = false;
  const bool used = tile_row(p, blk, q * 32 + lane) >= 0;
#pragma unroll 1
  for (int n0 = 0; n0 < NT; n0 += 32) {
    uint32_t w[32];
    tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + C::kCols + n0, w);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      bad |= n0 + i < NT && !(fabsf(__uint_as_float(w[i])) < INFINITY);
  }
  bad = __any_sync(0xffffffffu, bad && used);
  if (lane == 0) s_sum[warp] = bad;
  workers_sync();
  if ((s_sum[0] | s_sum[1] | s_sum[2] | s_sum[3]) == 0) return;
  Block<NT> f;
  bool run = true;
  const int blocks = (groups + 3) / 4;
  for (int j = rank, i = 0; j < blocks; j += S, ++i) {
    f.load_b(p, e, s_grp, j, groups, [&](int r) { return tile_row(p, blk, r); });
    f.store_b(p, e, smem);
    f.put_v(p, e, s_ad, t0, smem + C::kOffV);
    fence_proxy_async_smem();
    tc_fence_before();
    workers_sync();
    if (e == 0) {
      tc_fence_after();
      const uint64_t ad = sdesc_sw128(smem_u32(smem)), hi = sdesc_sw128(smem_u32(smem + C::kOffV)),
                     lo = sdesc_sw128(smem_u32(smem + C::kOffV + NT * 128));
      const int n = min(4, groups - 4 * j);
      for (int k = 0; k < n; ++k) {
        umma_bf16(tmem + C::kCols, ad + 2u * k, hi + 2u * k, idesc_bf16_f32(kRows, NT),
                  (i | k) != 0 ? 1u : 0u);
        umma_bf16(tmem + C::kCols, ad + 2u * k, lo + 2u * k, idesc_bf16_f32(kRows, NT), 1u);
      }
      umma_commit(redo);
    }
    int ok = 1;
    if (lane == 0 && run) ok = mbar_wait(redo, i & 1, s_abort) ? 1 : 0;
    if (lane == 0 && !ok) fail(s_abort, p.status);
    run = __shfl_sync(0xffffffffu, ok, 0) != 0 && run;
    tc_fence_after();
  }
}

template <int NT, bool SHRINK>
__global__ void __launch_bounds__(192, 1)
    lora_swap_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ CUtensorMap tmB, const LoraParams p) {
  using C = SwapCfg<NT, SHRINK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;    // the accumulators are complete
  uint64_t* tbl = tfull + 1;               // the groups are listed
  uint64_t* vfull = tfull + 2;             // a v tile is in its slot
  uint64_t* vempty = vfull + C::kVSlots;
  uint64_t* redo = vempty + C::kVSlots;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  int* s_total = reinterpret_cast<int*>(smem + C::kOffMisc + 12);
  int* s_sum = reinterpret_cast<int*>(smem + C::kOffMisc + 16);
  int* s_ad = reinterpret_cast<int*>(smem + C::kOffAd);
  uint32_t* s_grp = reinterpret_cast<uint32_t*>(smem + C::kOffGrp);
  float* part = reinterpret_cast<float*>(smem);           // [S][own tokens][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = gridDim.x, rank = blockIdx.x;
  const int t0 = blockIdx.z * NT;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tbl, 4);
    mbar_init(redo, 1);
    for (int s = 0; s < C::kVSlots; ++s) {
      mbar_init(&vfull[s], 4);
      mbar_init(&vempty[s], 1);
    }
    *s_abort = 0;
    if (!SHRINK) *s_total = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    if (!SHRINK) tma_prefetch_desc(&tmB);
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
  // SHRINK: blocks of eight groups.  How many there are is known here only: K is
  // split over as many of the cluster's CTAs as leave every block one turn.
  int split = S, unit = blockIdx.y, units = 1, turns_end = 1;
  if (SHRINK) {
    turns_end = (*s_total + 7) / 8;
    while (split > 1 && turns_end * split > S * static_cast<int>(gridDim.y)) split >>= 1;
    unit = static_cast<int>(blockIdx.y) * (S / split) + rank / split;
    units = static_cast<int>(gridDim.y) * (S / split);
  }
  const int part_of = rank & (split - 1);  // this CTA's part of K, and of the tokens
  const int per = NT / split;              // tokens of this CTA: a power of two
  const int kb0 = static_cast<int>(static_cast<long long>(KB) * part_of / split);
  const int kb1 = static_cast<int>(static_cast<long long>(KB) * (part_of + 1) / split);
  int stage = 0;
  uint32_t phase = 0, pass_parity = 0;
  for (int turn = 0; turn < turns_end; turn += units) {
    const int blk = turn + unit;
    const int ng = SHRINK ? min(8, *s_total - blk * 8) : 0;
    const bool idle = SHRINK && ng <= 0;
    if (warp == 0) {
      if (lane == 0 && !idle) {
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
        if (!SHRINK && ok && p.n > 0) {
          ok = mbar_wait(tbl, 0u, s_abort);
          const int total = ok ? *s_total : 0, blocks = (total + 3) / 4;
          for (int j = rank; ok && j < blocks; j += S) {
            if (!mbar_wait(&empty[stage], phase ^ 1u, s_abort)) {
              ok = false;
              break;
            }
            uint8_t* sa = smem + stage * C::kStage;
            const int n = min(4, total - 4 * j);
            mbar_expect_tx(&full[stage], static_cast<uint32_t>(n) * kRows * kGroup * 2);
            for (int g = 0; g < n; ++g) {
              const uint32_t gr = s_grp[4 * j + g];
              const int row = grp_adapter(gr) * p.N;
              uint8_t* to = sa + g * kRows * kGroup * 2;
              if (p.swiglu) {
                tma_load_2d(to, &tmB, &full[stage], grp_first(gr), row + blk * 64);
                tma_load_2d(to + kRows * kGroup, &tmB, &full[stage], grp_first(gr), row + p.outs + blk * 64);
              } else {
                tma_load_2d(to, &tmB, &full[stage], grp_first(gr), row + blk * kRows);
              }
            }
            if (++stage == C::kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok) {
          fail(s_abort, p.status);
          // the copies issued into the slots end before the CTA does
          for (int s = 0; s < C::kStages; ++s) mbar_wait(&full[s], s < stage ? phase : phase ^ 1u, nullptr);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0 && !idle) {
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
        if (!SHRINK && ok && p.n > 0) {
          ok = mbar_wait(tbl, 0u, s_abort);
          const int total = ok ? *s_total : 0, blocks = (total + 3) / 4;
          int sl = 0;
          uint32_t vphase = 0;
          for (int j = rank; ok && j < blocks; j += S) {
            if (!mbar_wait(&full[stage], phase, s_abort)) {
              ok = false;
              break;
            }
            const uint32_t sa = smem_u32(smem + stage * C::kStage);
            const int n = min(4, total - 4 * j);
            for (int k = 0; k < n; k += C::kG) {
              if (!mbar_wait(&vfull[sl], vphase, s_abort)) {
                ok = false;
                break;
              }
              tc_fence_after();
              uint32_t sv = smem_u32(smem + C::kOffV + sl * C::kVBytes);
              for (int g = k; g < k + C::kG && g < n; ++g, sv += 2 * C::kVTile) {
                // a group is one k-step for hi and one for lo
                const uint64_t ad = sdesc_sw32(sa + g * kRows * kGroup * 2);
                umma_bf16(tmem + C::kCols, ad, sdesc_sw32(sv), idesc, j != rank || g != 0 ? 1u : 0u);
                umma_bf16(tmem + C::kCols, ad, sdesc_sw32(sv + C::kVTile), idesc, 1u);
              }
              umma_commit(&vempty[sl]);
              if (++sl == C::kVSlots) {
                sl = 0;
                vphase ^= 1u;
              }
            }
            umma_commit(&empty[stage]);
            if (++stage == C::kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok) fail(s_abort, p.status);
        umma_commit(tfull);
        if (!ok) mbar_wait(tfull, pass_parity, nullptr);
      }
      __syncwarp();
    } else if (!SHRINK) {
      const int e = threadIdx.x - 64;
      if (p.n > 0) {
        // the adapters' indexes and ranks are inputs: read before v is there
        groups = build_groups<NT>(p, t0, e, s_ad, s_grp, s_sum);
        if (e == 0) *s_total = groups;
        __syncwarp();
        if (lane == 0) mbar_arrive(tbl);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        // a thread's values of the next slot are on their way while it waits for it
        constexpr int kG = C::kG;
        VRows<NT, kG> next;
        auto group_of = [&](int i) { return 4 * (rank + S * (i * kG >> 2)) + (i * kG & 3); };
        next.load(p, s_ad, s_grp, group_of(0), groups, t0, e);
        int sl = 0;
        uint32_t vphase = 0;
        for (int i = 0; group_of(i) < groups; ++i) {
          int ok = 1;
          if (lane == 0) ok = mbar_wait(&vempty[sl], vphase ^ 1u, s_abort) ? 1 : 0;
          if (!__shfl_sync(0xffffffffu, ok, 0)) {
            if (lane == 0) fail(s_abort, p.status);
            break;
          }
          next.store(smem + C::kOffV + sl * C::kVBytes, e);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&vfull[sl]);
          if (++sl == C::kVSlots) {
            sl = 0;
            vphase ^= 1u;
          }
          next.load(p, s_ad, s_grp, group_of(i + 1), groups, t0, e);
        }
      }
    }
    if (warp >= 2 && !idle) {
      int ok = 1;
      if (lane == 0) ok = mbar_wait(tfull, pass_parity, s_abort) ? 1 : 0;
      if (lane == 0 && !ok) fail(s_abort, p.status);
      __syncwarp();
      if (!SHRINK && 4 * rank < groups) look_over<NT>(p, smem, s_ad, s_grp, s_sum, redo, s_abort, tmem,
                                                      blk, t0, rank, S, groups, threadIdx.x - 64);
    }
    if (!idle) pass_parity ^= 1u;
    __syncwarp();
    if (split > 1) cluster_sync_all();   // every ring of the cluster is free
    // 1 << lg tokens a CTA sums; at: the place of the first CTA of this one's part of
    // the cluster (constants for SHRINK, whose split the compiler cannot tell)
    auto push = [&](int lg, int at) {
      tc_fence_after();
      const int q = warp & 3;
      const uint32_t mine = smem_u32(part) + static_cast<uint32_t>((part_of * per * kRows + q * 32 + lane) * 4);
#pragma unroll 1
      for (int n0 = 0; n0 < NT && t0 + n0 < p.T; n0 += 32) {
        uint32_t v[32];
        unsigned wanted = 0xffffffffu;
        if (SHRINK) {      // a warp has two groups: only their adapters' tokens
          const int g = 2 * q, n = n0 + lane, a = n < NT ? s_ad[n] : -1;
          const uint32_t* grp = s_grp + blk * 8;
          wanted = __ballot_sync(0xffffffffu, a >= 0 && ((g < ng && a == grp_adapter(grp[g])) ||
                                                         (g + 1 < ng && a == grp_adapter(grp[g + 1]))));
          if (wanted == 0u) continue;
        }
        tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + n0, v);
        if (!SHRINK && 4 * rank < groups) {      // this CTA had adapter k-blocks
          uint32_t w[32];
          tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + C::kCols + n0, w);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
        }
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int n = n0 + i;
          if (n < NT && t0 + n < p.T && (wanted >> i & 1u))
            st_cluster_f32(mapa_shared(mine + static_cast<uint32_t>((n & ((1 << lg) - 1)) * kRows * 4),
                                       static_cast<uint32_t>(at + (n >> lg))),
                           __uint_as_float(v[i]));
        }
      }
      tc_fence_before();
    };
    // SHRINK with all of K here: the sums are v
    auto direct = [&]() {
      tc_fence_after();
      const int q = warp & 3;
      const ShrinkRow m(p, s_grp + blk * 8, ng, q * 32 + lane);
#pragma unroll 1
      for (int n0 = 0; n0 < NT && t0 + n0 < p.T; n0 += 32) {
        const unsigned mine = m.tokens(n0 + lane < NT ? s_ad[n0 + lane] : -1);
        const unsigned any = __reduce_or_sync(0xffffffffu, mine);
        if (any == 0u) continue;
        uint32_t v[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + n0, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if ((any >> i & 1u) && (mine >> i & 1u)) m.put(p, t0 + n0 + i, __uint_as_float(v[i]));
      }
      tc_fence_before();
    };
    if (warp >= 2 && !idle) {
      constexpr int kLg = NT == 256 ? 8 : NT == 128 ? 7 : NT == 64 ? 6 : NT == 32 ? 5 : 4;
      if (SHRINK && split == 1)
        direct();
      else if (!SHRINK || split == S)
        push(31 - __clz(NT / S), 0);
      else if (split == 4)
        push(kLg - 2, rank & ~3);
      else
        push(kLg - 1, rank & ~1);
    }
    __syncwarp();
    if (split > 1)
      cluster_sync_all();
    else
      __syncthreads();
    if (warp >= 2 && !idle && !(SHRINK && split == 1)) {
      const int lr = (warp & 3) * 32 + lane, first = t0 + part_of * per, count = min(per, p.T - first);
      const int* ad = s_ad + part_of * per;
      const uint32_t* grp = s_grp + (SHRINK ? blk * 8 : 0);
      switch (split) {
        case 1: finish<SHRINK, 1>(p, part, ad, grp, ng, first, count, per, blk, lr); break;
        case 2: finish<SHRINK, 2>(p, part, ad, grp, ng, first, count, per, blk, lr); break;
        case 4: finish<SHRINK, 4>(p, part, ad, grp, ng, first, count, per, blk, lr); break;
        default: finish<SHRINK, 8>(p, part, ad, grp, ng, first, count, per, blk, lr); break;
      }
    }
    if (SHRINK) {
      fence_proxy_async_smem();   // the next block's copies land where the sums were
      __syncthreads();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// ---------------------------------------------------------------- CTA pairs, many tokens
// 256 tokens x 256 rows of W a tile (tcgen05 cta_group::2: each CTA holds 128
// token rows and half of the weight rows), persistent, accumulators double
// buffered in TMEM so that a tile's stores run under the next tile's MMAs.
// Warps: 0 TMA, 1 MMA (leader), 2-5 stores, 6-9 adapters' groups.  The last run
// ahead, and the MMA warp takes a group after each k-block of a tile's second
// half, so that their slots' round trips lie under the K columns; always there,
// whatever is ready, so that the order of the sums does not change.
// Bound: the tensor cores.  16384 tokens, K 7168, N 4096: 608 us without adapters
// (1.58 PFLOP/s, power capped), 672 with 32 of up to rank 64, of which v is 45.
// 1024 tokens with an adapter each: 43 and 162, a group's slot 0.5 us.
constexpr int kPairN = 256;
constexpr int kPairStages = 5;
constexpr int kPairSlots = 3;                                     // groups of adapter columns under way
constexpr int kPairThreads = 192 + kWorkers;
constexpr uint32_t kPairTmem = 2 * kPairN;

struct PairCfg {
  static constexpr uint32_t kStage = 2 * kTile;                   // 128 token rows, 128 W rows
  static constexpr uint32_t kGroupTile = kRows * kGroup * 2;
  static constexpr uint32_t kSlot = 3 * kGroupTile;               // v's hi and lo, the factors
  static constexpr uint32_t kOffSlot = kPairStages * kStage;
  static constexpr uint32_t kOffOut = kOffSlot + kPairSlots * kSlot;
  static constexpr uint32_t kOffBar = kOffOut + 4 * kStageRowsBytes;
  static constexpr uint32_t kOffMisc = kOffBar + (2 * kPairStages + 2 * kPairSlots + 5) * 8;
  static constexpr uint32_t kOffAd = kOffMisc + 64;
  static constexpr uint32_t kOffGrp = kOffAd + kMaxTileTokens * 4;
  static constexpr uint32_t kUsed = kOffGrp + kMaxTileTokens * 8 * 4;
  static constexpr uint32_t kSmem = kUsed + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint64_t t0 = 0;
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
    if (t0 == 0) t0 = globaltimer();
    if (globaltimer() - t0 > kWaitLimitNs) return false;
  }
}

__device__ __forceinline__ void arrive_release_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// A worker's factor row and token row of one group of adapter columns.
struct PairRow {
  uint4 b0, b1;
  float4 v[4];
  int cols, first;
  bool own;
};

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
  uint64_t* lempty = lfull + kPairSlots;
  uint64_t* tfull = lempty + kPairSlots;
  uint64_t* tempty = tfull + 2;            // leader
  uint64_t* done = tempty + 2;             // leader
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* s_more = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  int* s_sum = reinterpret_cast<int*>(smem + C::kOffMisc + 32);
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
    for (int s = 0; s < kPairSlots; ++s) {
      mbar_init(&lfull[s], 8);
      mbar_init(&lempty[s], 1);
    }
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
      int stage = 0, acc = 0, slot = 0;
      uint32_t phase = 0, aphase = 0, lp = 0;
      bool ok = true, more = false;
      // one group of the tile's adapter columns; the slot that ends them holds none
      auto take = [&](uint32_t d) {
        if (!mbar_wait_cluster(&lfull[slot], lp, s_abort)) {
          ok = false;
          return;
        }
        more = s_more[slot] != 0;
        if (more) {
          tc_fence_after();
          const uint32_t at = smem_u32(smem + C::kOffSlot + slot * C::kSlot);
          const uint64_t b = sdesc_sw32(at + 2 * C::kGroupTile);
          umma_bf16_pair(d, sdesc_sw32(at), b, idesc, 1u);
          umma_bf16_pair(d, sdesc_sw32(at + C::kGroupTile), b, idesc, 1u);
        }
        umma_commit_pair(&lempty[slot], 0x3);
        if (++slot == kPairSlots) {
          slot = 0;
          lp ^= 1u;
        }
      };
      for (int w = cid; ok && w < total; w += ncl) {
        if (!mbar_wait(&tempty[acc], aphase ^ 1u, s_abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * kPairN);
        more = true;
        for (int kb = 0; ok && kb < KB; ++kb) {
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
          if (more && 2 * kb >= KB) take(d);
        }
        while (ok && more) take(d);
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
                silu_fast(__uint_as_float(gv[2 * i])) * __uint_as_float(uv[2 * i]),
                silu_fast(__uint_as_float(gv[2 * i + 1])) * __uint_as_float(uv[2 * i + 1]));
        } else {
          uint32_t v[32];
          tmem_ld32(tbase + ci * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        }
        const int col = nt * per_n + ci * 32, col0 = col - (ci & 1) * 32;
        if (p.vec_y == 16 && (ci & 1) == 0) {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
        }
        // the map clips rows, and columns in pieces of 16 bytes only: what lies behind
        // an end inside such a piece would be written
        if (p.vec_y == 16 && ((p.outs & 7) == 0 || col0 + 64 <= p.outs)) {
          stage_row_32(sbuf, lane, (ci & 1) * 4, pk);
          if ((ci & 1) != 0) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (row0 < p.T && col0 < p.outs) tma_store_2d(&tmY, sbuf, col0, row0);
              bulk_commit();
            }
          }
        } else {
          // rows the map cannot describe, and their ends: through the buffer, so that
          // a warp stores 64 neighbouring columns of a row at a time
          stage_row_32(sbuf, lane, (ci & 1) * 4, pk);
          if ((ci & 1) != 0) {
            __syncwarp();
            const int c0 = col0 + lane, c2 = col0 + 2 * lane;
            const int rows = min(32, p.T - row0);
            if (p.vec_y >= 4) {
              const uint8_t* from = sbuf + ((lane & 3) << 2);
              if (c2 + 1 < p.outs) {
#pragma unroll 4
                for (int r = 0; r < rows; ++r)
                  *reinterpret_cast<uint32_t*>(p.y + (row0 + r) * p.ldy + c2) =
                      *reinterpret_cast<const uint32_t*>(from + r * 128 + (((lane >> 2) ^ (r & 7)) << 4));
              } else if (c2 < p.outs) {     // the last of an odd number
                for (int r = 0; r < rows; ++r)
                  p.y[(row0 + r) * p.ldy + c2] =
                      *reinterpret_cast<const __nv_bfloat16*>(from + r * 128 + (((lane >> 2) ^ (r & 7)) << 4));
              }
            } else {
#pragma unroll 4
              for (int r = 0; r < 32 && row0 + r < p.T; ++r) {
                const __nv_bfloat16* from = reinterpret_cast<const __nv_bfloat16*>(sbuf + r * 128);
                __nv_bfloat16* dst = p.y + (row0 + r) * p.ldy;
                // element k of row r: chunk k / 8 at (k / 8) ^ (r % 8)
                const int lo = (((lane >> 3) ^ (r & 7)) << 3) + (lane & 7);
                const int hi = ((((lane >> 3) + 4) ^ (r & 7)) << 3) + (lane & 7);
                if (c0 < p.outs) dst[c0] = from[lo];
                if (c0 + 32 < p.outs) dst[c0 + 32] = from[hi];
              }
            }
            __syncwarp();
          }
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
    bool waited = p.wait_first != 0;
    uint32_t lp = 0;
    int built = -1, groups = 0, slot = 0;
    unsigned dirty = (1u << kPairSlots) - 1u;   // slots whose row of v is not zero
    bool run = true;   // after a wait that gave up: keep the workers' barriers, touch nothing
    // where row e's two chunks of 16 bytes lie under the 32-byte swizzle
    const uint32_t c0 = static_cast<uint32_t>(e) * 32u + ((static_cast<uint32_t>(e) & 4u) << 2);
    for (int w = cid; w < total; w += ncl) {
      const int mt = w / n_tiles, nt = w - mt * n_tiles;
      if (mt != built) {
        workers_sync();                    // the last tile's table is no longer read
        groups = build_groups<kMaxTileTokens>(p, mt * 256, e, s_ad, s_grp, s_sum);
        built = mt;
      }
      const int half = p.swiglu ? 64 : kRows;
      const int o = nt * per_n + static_cast<int>(rank) * half + (e < half ? e : e - half);
      const int wr = o < p.outs ? (e < half ? o : p.outs + o) : -1;
      const int t = mt * 256 + static_cast<int>(rank) * 128 + e;
      const int mine = s_ad[static_cast<int>(rank) * 128 + e];   // -1 past the last token
      const __nv_bfloat16* brow = p.b + static_cast<long long>(wr) * p.r_max;
      const float* vrow = p.v + static_cast<long long>(t) * p.r_max;
      // this thread's factor row and token row of the next groups: as many as
      // there are slots, all on their way together, because what makes a slot's
      // contents visible waits for every load before it
      PairRow ahead[kPairSlots];
      auto load_b = [&](PairRow& f, int j) {
        const uint32_t g = j < groups ? s_grp[j] : 0u;
        f.cols = j < groups ? grp_cols(g) : 0;
        f.first = grp_first(g);
        f.own = j < groups && grp_adapter(g) == mine;
        f.b0 = f.b1 = make_uint4(0u, 0u, 0u, 0u);
        if (f.cols > 0 && wr >= 0) {
          const uint4* b = reinterpret_cast<const uint4*>(
              brow + static_cast<long long>(grp_adapter(g)) * p.N * p.r_max + f.first);
          f.b0 = __ldg(b);
          if (f.cols > 8) f.b1 = __ldg(b + 1);
        }
      };
      auto load_v = [&](PairRow& f) {
        if (!f.own) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f.v[i] = 8 * (i / 2) < f.cols ? __ldcg(reinterpret_cast<const float4*>(vrow + f.first) + i)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
      };
#pragma unroll
      for (int i = 0; i < kPairSlots; ++i) load_b(ahead[i], i);
      if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
      waited = true;
#pragma unroll
      for (int i = 0; i < kPairSlots; ++i) load_v(ahead[i]);
      // the post after the last group ends the tile
      for (int j0 = 0; run && j0 <= groups; j0 += kPairSlots) {
        const int n = min(kPairSlots, groups + 1 - j0), first = slot;
#pragma unroll
        for (int i = 0; i < kPairSlots; ++i) {
          if (!run || i >= n) break;
          const PairRow& f = ahead[i];
          int ok = 1;
          if (lane == 0) ok = mbar_wait(&lempty[slot], lp ^ 1u, s_abort) ? 1 : 0;
          run = __shfl_sync(0xffffffffu, ok, 0) != 0;
          if (!run) {
            if (lane == 0) fail(s_abort, p.status);
            break;
          }
          if (j0 + i < groups) {
            uint8_t* at = smem + C::kOffSlot + slot * C::kSlot + c0;
            uint8_t* at1 = smem + C::kOffSlot + slot * C::kSlot + (c0 ^ 16u);
            bool bad = false;
            *reinterpret_cast<uint4*>(at + 2 * C::kGroupTile) = clean8(f.b0, f.cols, bad);
            *reinterpret_cast<uint4*>(at1 + 2 * C::kGroupTile) = clean8(f.b1, f.cols - 8, bad);
            if (bad) report(p.status, MOE_ERR_NONFINITE);
            if (f.own || (dirty >> slot & 1u)) {
              uint4 hi0 = make_uint4(0u, 0u, 0u, 0u), lo0 = hi0, hi1 = hi0, lo1 = hi0;
              if (f.own) {
                split8(f.v[0], f.v[1], hi0, lo0);
                split8(f.v[2], f.v[3], hi1, lo1);
              }
              *reinterpret_cast<uint4*>(at) = hi0;
              *reinterpret_cast<uint4*>(at + C::kGroupTile) = lo0;
              *reinterpret_cast<uint4*>(at1) = hi1;
              *reinterpret_cast<uint4*>(at1 + C::kGroupTile) = lo1;
              dirty = f.own ? dirty | 1u << slot : dirty & ~(1u << slot);
            }
          }
          if (e == 0) s_more[slot] = j0 + i < groups ? 1 : 0;
          if (++slot == kPairSlots) {
            slot = 0;
            lp ^= 1u;
          }
        }
        if (!run) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          for (int i = 0; i < n; ++i) {
            const int at = first + i < kPairSlots ? first + i : first + i - kPairSlots;
            arrive_release_cluster(lfull_l + 8u * static_cast<uint32_t>(at));
          }
        }
#pragma unroll
        for (int i = 0; i < kPairSlots; ++i) load_b(ahead[i], j0 + kPairSlots + i);
#pragma unroll
        for (int i = 0; i < kPairSlots; ++i) load_v(ahead[i]);
      }
    }
    // the last commits on this CTA's lempty have arrived
    for (int i = 0; run && i < kPairSlots; ++i) {
      if (lane == 0 && !mbar_wait(&lempty[slot], lp ^ 1u, nullptr)) fail(s_abort, p.status);
      if (++slot == kPairSlots) {
        slot = 0;
        lp ^= 1u;
      }
    }
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

// Tokens per tile, splits of K and kernel, by an estimate of the time in us:
// rounds of CTAs x k-blocks x the slowest of
//   the weight tiles' way from HBM (16 KB per CTA, shared by the token tiles),
//   the bytes into an SM (120 GB/s each measured with all SMs at it),
//   the MMA (0.33 us for 128 x 256 x 64 in one CTA; less falls slower than N)
// plus what a CTA does before and after its loop, which grows with its tokens
// and, for the cluster's exchange of partial sums, with them again.  How many
// adapters meet in a tile is known on the device only: the estimate is the
// geometric mean of none and of as many as there can be, each of whose groups
// of columns costs a slot (0.15 us at 16 tokens to 0.6 at 256, over the splits).
// Swapped against pairs, K 7168, N 4096, 48 adapters of r 32 a token each, then in
// requests of 64, then none: 512 tokens 85, 41, 39 and 142, 53, 46 us; 1024 148, 75, 63
// and 162, 72, 47; 2048 279, 129, 120 and 298, 109, 84.  The estimate takes the
// swapped kernel up to 512, pairs from 768.
struct Shape {
  int nt, splits;      // nt = 0: CTA pairs
};

// CTAs that run at a time in clusters of S, a CTA a SM: the parts of the chip
// that a cluster must fit into are no multiples of it (152 SMs: 144 of four,
// 120 of eight; 128 CTAs in clusters of eight took two rounds, 14 us where
// fours took 9.5).  Asked once.
int cluster_room(int S, int sm) {
  static std::atomic<int> known[64][4];
  if (S == 1) return sm;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sm;
  std::atomic<int>& k = known[dev][S == 2 ? 1 : (S == 4 ? 2 : 3)];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    using C = SwapCfg<256, true>;
    auto kern = lora_swap_kernel<256, true>;
    static bool done[64] = {false};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S);
    cfg.blockDim = dim3(192);
    cfg.dynamicSmemBytes = C::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (set_smem_once(kern, static_cast<int>(C::kSmem), done) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return sm / S * S;
    }
    n *= S;
    k.store(n, std::memory_order_relaxed);
  }
  return n < sm ? n : sm;
}

Shape pick_shape(int T, int K, int outs, int rows_per_tile, int adapters, int r_max, int sm) {
  const double KB = (K + kBK - 1) / kBK;
  Shape best{0, 1};
  const double pair_tiles = static_cast<double>((T + 255) / 256) * ((outs + 2 * rows_per_tile - 1) / (2 * rows_per_tile));
  const double pairs = sm > 1 ? sm / 2 : 1;
  const double groups = r_max / 32.0 + 0.5;          // of an adapter, ranks being mixed
  auto both = [](double us, double more) { return std::sqrt(us * (us + more)); };
  const double pair_rounds = std::ceil(pair_tiles / pairs);
  double least = both(pair_rounds * KB * 0.33 + 6.0, pair_rounds * 0.5 * groups * std::min(adapters, 256));
  const int rows = (outs + rows_per_tile - 1) / rows_per_tile;
  for (int nt = 16; nt <= 256; nt *= 2) {
    const int tt = (T + nt - 1) / nt;
    if (tt > 64) continue;
    for (int S = 1; S <= 8 && S <= KB; S *= 2) {
      const double ctas = static_cast<double>(rows) * tt * S;
      const int room = cluster_room(S, sm);
      const double rounds = std::ceil(ctas / room), busy = ctas < room ? ctas : room;
      const double hbm = 16384.0 * busy / tt / 7.0e6, in = (16384.0 + 128.0 * nt) / 1.2e5;
      const double mma = 0.12 + nt * 0.0008;
      const double block = hbm > in ? (hbm > mma ? hbm : mma) : (in > mma ? in : mma);
      const double us = rounds * (std::ceil(KB / S) * block + 3.0 + nt * 0.01 +
                                  (S > 1 ? 0.8 + nt * 0.015 : 0.0));
      const double est = both(us, rounds * (0.12 + nt * 0.0018) * groups * std::min(adapters, nt) / S);
      if (est < least) {
        least = est;
        best = Shape{nt, S};
      }
    }
  }
  return best;
}

// Tokens per tile where the factors of A are the rows.  A tile's sums take as
// long as its loads where there are few blocks of eight groups, so half a tile
// is faster up to three (691 tokens, K 5048, 6 adapters, r 32: 18 and 23 us);
// with more, x is read again for each (512 tokens, K 7168, 48 adapters: 98 and 85).
int tile_tokens(int T, int adapters, int r_max) {
  const int groups = std::min(adapters, 256) * ((r_max + kGroup - 1) / kGroup);
  const int most = groups <= 3 * 8 && T <= 128 * 65535 ? 128 : 256;   // 65535: a grid's z
  int nt = 16;
  while (nt < T && nt < most) nt *= 2;
  return nt;
}

// Up to tokens x r_max x (K + 5000) v is a dot product per token and rank: every
// row of A is read from L2 for each of its tokens, the tensor cores' kernel reads
// it once a tile and takes 8 us for the least.
constexpr double kDotMost = 1e8;

// bf16, encoded anew on every call: x, y and their strides are the caller's.
bool encode_tmap_bf16(CUtensorMap* m, const void* base, long long rows, int cols, long long ld, int box_rows,
                      int box_cols = 64) {
  return encode_tmap(m, base, 2, rows, cols, ld, box_rows, box_cols);
}

template <int NT, bool SHRINK>
cudaError_t run_swap(const LoraArgs& g, const LoraParams& p, int S, cudaStream_t s) {
  using C = SwapCfg<NT, SHRINK>;
  CUtensorMap tw, tx, tb;
  if (SHRINK) {
    if (!encode_tmap_bf16(&tw, g.a, static_cast<long long>(g.n_adapters) * g.r_max, g.K, g.K, kGroup))
      return cudaErrorInvalidValue;
  } else if (!encode_tmap_bf16(&tw, g.w, g.N, g.K, g.K, g.swiglu ? 64 : kRows)) {
    return cudaErrorInvalidValue;
  }
  if (!encode_tmap_bf16(&tx, g.x, g.T, g.K, g.ldx, NT)) return cudaErrorInvalidValue;
  if (SHRINK || g.n_adapters == 0)
    tb = tx;                              // not used
  else if (!encode_tmap_bf16(&tb, g.b, static_cast<long long>(g.n_adapters) * g.N, g.r_max, g.r_max,
                             g.swiglu ? 64 : kRows, kGroup))
    return cudaErrorInvalidValue;
  const int KB = (g.K + kBK - 1) / kBK;
  const int tt = (g.T + NT - 1) / NT;
  int rows;                               // blocks of 128 rows
  if (SHRINK) {
    // how many blocks a tile has is known on the device only: the widest
    // clusters that leave not too many SMs without one, and the blocks share
    // them out between K and themselves
    const long long adapters = g.n_adapters < NT ? g.n_adapters : NT;
    const long long most = (adapters * ((g.r_max + kGroup - 1) / kGroup) + 7) / 8;
    auto rows_at = [&](int c) {
      return std::min(most, std::max<long long>(1, cluster_room(c, g.sm_count) / (static_cast<long long>(tt) * c)));
    };
    long long used = 0;
    // up to four k-blocks one CTA takes them all (K 136: 15.4 us, split 19.7; K 512 18, 14)
    for (int c = 1; c <= 8 && (c == 1 || KB > 4) && c <= KB; c *= 2) {
      if (static_cast<long long>(tt) * c > cluster_room(c, g.sm_count)) break;
      used = std::max(used, tt * c * rows_at(c));
      if (5 * tt * c * rows_at(c) >= 3 * used) S = c;
    }
    rows = static_cast<int>(rows_at(S));
  } else {
    const int per = g.swiglu ? 64 : kRows;
    rows = (p.outs + per - 1) / per;
  }
  auto kern = lora_swap_kernel<NT, SHRINK>;
  static bool done[64] = {false};
  const cudaError_t e = set_smem_once(kern, static_cast<int>(C::kSmem), done);
  if (e != cudaSuccess) return e;
  return launch_cluster(kern, dim3(S, rows, tt), 192, static_cast<int>(C::kSmem), S, s, tw, tx, tb, p);
}

cudaError_t run_shrink(const LoraArgs& g, const LoraParams& p, int tile, cudaStream_t s) {
  switch (tile) {
    case 16: return run_swap<16, true>(g, p, 1, s);
    case 32: return run_swap<32, true>(g, p, 1, s);
    case 64: return run_swap<64, true>(g, p, 1, s);
    case 128: return run_swap<128, true>(g, p, 1, s);
    default: return run_swap<256, true>(g, p, 1, s);
  }
}

cudaError_t run_project(const LoraArgs& g, const LoraParams& p, Shape shape, cudaStream_t s) {
  switch (shape.nt) {
    case 16: return run_swap<16, false>(g, p, shape.splits, s);
    case 32: return run_swap<32, false>(g, p, shape.splits, s);
    case 64: return run_swap<64, false>(g, p, shape.splits, s);
    case 128: return run_swap<128, false>(g, p, shape.splits, s);
    default: return run_swap<256, false>(g, p, shape.splits, s);
  }
}

cudaError_t run_pair(const LoraArgs& g, const LoraParams& p, cudaStream_t s) {
  CUtensorMap tx, tw, ty;
  if (!encode_tmap_bf16(&tx, g.x, g.T, g.K, g.ldx, 128)) return cudaErrorInvalidValue;
  if (!encode_tmap_bf16(&tw, g.w, g.N, g.K, g.K, g.swiglu ? 64 : 128)) return cudaErrorInvalidValue;
  if (p.vec_y != 16)
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

size_t lora_workspace_bytes(int T, int r_max) { return static_cast<size_t>(T) * r_max * 4; }

LoraPlan lora_plan(const LoraArgs& g) {
  const Shape shape = pick_shape(g.T, g.K, g.swiglu ? g.N / 2 : g.N, g.swiglu ? 64 : kRows, g.n_adapters, g.r_max,
                                 g.sm_count);
  const bool dots = static_cast<double>(g.T) * g.r_max * (g.K + 5000.0) <= kDotMost;
  return LoraPlan{shape.nt, shape.splits, dots ? 0 : tile_tokens(g.T, g.n_adapters, g.r_max)};
}

cudaError_t launch_lora_project(const LoraArgs& g, cudaStream_t s) {
  LoraParams p{};
  p.b = static_cast<const __nv_bfloat16*>(g.b);
  p.ranks = g.ranks;
  p.scales = g.scales;
  p.adapter = g.adapter;
  p.v = static_cast<float*>(g.ws);
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
  const LoraPlan plan = lora_plan(g);
  if (g.n_adapters > 0) {
    cudaError_t e;
    if (plan.v_tile == 0)
      e = launch_pdl(lora_dot_kernel, dim3(g.r_max / kDotRanks, g.T), dim3(kDotThreads), 0, s, p,
                     static_cast<const __nv_bfloat16*>(g.x), static_cast<const __nv_bfloat16*>(g.a),
                     g.ldx);
    else
      e = run_shrink(g, p, plan.v_tile, s);
    if (e != cudaSuccess) return e;
  }
  if (plan.tile != 0) return run_project(g, p, Shape{plan.tile, plan.splits}, s);
  const uintptr_t at = reinterpret_cast<uintptr_t>(g.y);
  p.vec_y = (at & 15u) == 0 && g.ldy % 8 == 0 ? 16 : ((at & 3u) == 0 && g.ldy % 2 == 0 ? 4 : 2);
  return run_pair(g, p, s);
}

}  // namespace moe
