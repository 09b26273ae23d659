// Products of bf16 rows with packed 4-bit weights, dense or grouped by expert, on
// the tensor cores: y_r = x_r W^T, or with SwiGLU silu(x_r G^T) * (x_r U^T).
//
// 128 rows of weights are the M side of tcgen05.mma, a chunk of up to NT tokens the
// N side, so every weight is expanded once per chunk.  The expanded weights never
// see shared memory: a thread reads one row's codes of 128 inputs (four 16-byte
// loads), expands them in registers (quant.cuh) and stores them as the A operand in
// TMEM; only the tokens come from shared memory.  Expanding into shared memory
// instead would write and read 2 bytes a weight there, four times the codes' own
// traffic and more than an SM's 128 bytes a clock carry at the rate HBM delivers
// codes.
//
// An item is two 128-row tiles (of one matrix, or the gate and up rows of the same
// 128 features) x one chunk of a group's tokens, the whole of K: both tiles share
// the chunk's tokens, halving their traffic.
// Roles of the warps, one CTA an SM, items dealt round robin:
//   0       bulk copies of weight records (128 inputs of both tiles) into a ring
//   1, 22   MMA issue, a tile each, so that one's waits pass under the other's MMAs
//           (warp 1 has the TMEM, too)
//   2-5     epilogue (TMEM lane quarter = warp % 4)
//   6-21    expansion: four warps a tile, for every other record
//   23(-26) token rows into a ring of their own: by TMA, or GATHER: copies of the
//           rows that an index names
// The two rings free a record as soon as its codes are in registers; two records'
// TMEM buffers let one be expanded while the last one multiplies.
// Every wait is bounded.
//
// Measured on a GB300, calls in a graph: 64 tokens of K 7168, N 4096 12.5 us, 16384 tokens
// 557 (1.73 PFLOP/s; call by call for long 620, as the power cap lowers the clock);
// a layer of 64 tokens on 32 units of 3584 180 us (4.17 TB/s), experts of 1024 and 8192
// tokens (128 of 768, k 8) 128 and 581.  When these took 185, 134 and 593, 169, 116 and 500
// were left without the MMAs, 159, 109 and 531 without the expansion's arithmetic, 147, 96
// and 438 without either: issue slots (72% busy) and the wait for a record's stores,
// barriers and MMAs bound the first two, the rows' way from L2 (about 10 TB/s) and the one
// set of accumulators of a wide chunk the last.
#include <algorithm>
#include <type_traits>

#include "gemm_common.cuh"
#include "moe_internal.h"
#include "quant.cuh"

namespace moe {
namespace {

constexpr int kExpandWarps = 16;
constexpr int kMmaWarp = 6 + kExpandWarps;        // of the second tile
constexpr int kTokenWarp = kMmaWarp + 1;
constexpr int kGatherThreads = 128;
constexpr int kThreads = (kTokenWarp + 1) * 32;
constexpr int kThreadsGather = kTokenWarp * 32 + kGatherThreads;
constexpr int kHalf = 64;                         // inputs of a block of a token stage
constexpr int kMaxSplits = 8;                     // CTAs of a cluster
constexpr uint32_t kMaxRecord = quant_record(16);
constexpr uint32_t kWStage = 2 * kMaxRecord;      // both tiles' records of 128 inputs
// TMEM buffers of expanded weights, a record each (a tile's columns, then the other's).  Halves
// of a record let its MMAs start earlier, but take twice the barriers (layer of 64 tokens 218
// us, 183 so; 16384 tokens of K 7168, N 4096 575, 573).
constexpr int kABufs = 2;
constexpr uint32_t kACols = 128;
constexpr uint32_t kTmemD = kABufs * kACols;      // the accumulators' first column

// Columns of a chunk that each of `splits` CTAs sums: even, and splits times it covers
// the 16s that the rows fill.
__host__ __device__ constexpr int columns_of(int rows, int splits) {
  return ((rows + 15) / 16 * 16 + 2 * splits - 1) / (2 * splits) * 2;
}
constexpr int most_columns(int nt) {       // all CTAs' together
  int m = 0;
  for (int s = 2; s <= kMaxSplits; ++s) m = std::max(m, s * columns_of(nt, s));
  return m;
}

template <int NT, bool SPLIT>
struct TileCfg {
  // Records in flight, even, and token stages of 128 inputs (layer of 64 tokens 180.0 us, 180.9
  // with 6 and 4, 183.7 with 8 and 4; chunks of 128: 8192 tokens 583, with 6 and 3 594).
  static constexpr int kW = 4;
  static constexpr int kB = SPLIT || NT == 128 ? 4 : 6;
  static constexpr uint32_t kTok = NT * kQK * 2;
  static constexpr uint32_t kOffW = kB * kTok;
  static constexpr uint32_t kOffPart = kOffW + kW * kWStage;
  static constexpr uint32_t kPart = SPLIT ? most_columns(NT) * 256 * 4 : 0;
  static constexpr uint32_t kOffBar = kOffPart + kPart;
  static constexpr int kDBufs = NT == 128 ? 1 : 2;
  static constexpr int kBars = 2 * kW + 2 * kB + 2 * kABufs + 2 * kDBufs + 1;
  static constexpr uint32_t kOffMisc = kOffBar + kBars * 8;
  static constexpr uint32_t kOffOut = (kOffMisc + 16 + 127) / 128 * 128;   // 1 KB an epilogue warp
  static constexpr uint32_t kOffPrefix = kOffOut + 4 * 1024;
  static constexpr uint32_t kOffOffs = kOffPrefix + (kMaxGroups + 1) * 4;
  static constexpr uint32_t kSmem = kOffOffs + (kMaxGroups + 1) * 4 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kTmemD + kDBufs * 2 * NT <= 512, "TMEM columns");
};

struct TileParams {
  const uint8_t* w;
  const float* factor;
  const uint4* x;              // GATHER
  const int32_t* token;
  const int32_t* offsets;
  void* out;
  long long ldx, ldo, out_rows;
  size_t matrix;
  uint32_t record;
  int n_groups, dense_rows, x_rows, n, K, kb, rt, blocks, code, group, swiglu, f32, vec, early, splits;
  int32_t* status;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 16 lanes x 16 fp32 columns: thread i has lanes i / 4 (r[0], r[1] and r[4], r[5]) and
// i / 4 + 8, columns 2 (i % 4) and the next of each block of eight.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
      : "r"(taddr));
}

// Four 8x8 blocks of bf16, transposed: a row of the block that lane i names gets column
// i % 8 of block i / 8.
__device__ __forceinline__ void stmatrix_trans(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// SiLU by the approximate exponential and reciprocal: within (4 + 1.2 |g|) 2^-23 of its
// value (0 below -87), far below the bf16 that it is rounded to.
__device__ __forceinline__ float silu_fast(float g) { return __fdividef(g, 1.f + __expf(-g)); }

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T over 64 inputs, four MMAs: lane = row of A, a column
// two consecutive bf16 inputs.  Called by a whole warp, which elects the issuing lane
// here: under a branch that one lane takes, the operands are not uniform, and an MMA
// took 47 clocks to issue in a probe and 107 among this kernel's busy warps, whatever
// N; so it takes what it executes in, 14 at N 16, 32 at 64, 64 at 128.
__device__ __forceinline__ void umma_bf16_ts64(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Barriers by their shared-memory address.
__device__ __forceinline__ bool try_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// umma_commit by a whole warp.  The lane elected is the same at every call.
__device__ __forceinline__ void commit_at(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// mbar_wait's loop.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = globaltimer();
  while (true) {
    for (int i = 0; i < 64; ++i)
      if (try_wait_at(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > kWaitLimitNs) return false;
  }
}

// A wait of a whole warp; false where one of its lanes gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, try_wait_at(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_on(bar, parity, abort));
}

// A value that all lanes have, in a uniform register: what an MMA's operands and the
// loops around it are made of has to be there, or each MMA pays for moving it.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// 64 expanded weights of a row (pieces c[0] and c[1]; s2: their scale bytes) to TMEM
// columns d .. d + 31.
template <int CODE>
__device__ __forceinline__ void expand_half(const uint4& c0, const uint4& c1, uint32_t bytes, uint32_t d) {
  uint32_t v[32];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4& c = i == 0 ? c0 : c1;
    const uint32_t word[4] = {c.x, c.y, c.z, c.w};
    using Scale = QuantScale<CODE>;
    Scale q[2];
    q[0] = i == 0 ? Scale::template at<0>(bytes) : Scale::template at<2>(bytes);
    q[1] = i == 0 ? Scale::template at<1>(bytes) : Scale::template at<3>(bytes);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t e[4];
      quant_expand<CODE>(word[w], q[w >> 1], e);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[16 * i + 4 * w + j] = e[j];
    }
  }
  tmem_st32(d, v);
}

// Next slot of a ring of n, with the phase that a wait on its barrier goes by.
__device__ __forceinline__ void advance(int& slot, uint32_t& phase, int n) {
  if (++slot == n) {
    slot = 0;
    phase ^= 1u;
  }
}

// 768 threads leave 80 registers each, 864 with the gathering warps 72.  Of the three ungathered
// variants the two that do not split spill 72 bytes a thread (124 of loads).
template <int NT, bool GATHER, bool SPLIT>
__global__ void __launch_bounds__(GATHER ? kThreadsGather : kThreads, 1)
    quant_tile_kernel(const __grid_constant__ CUtensorMap tm16,
                      const __grid_constant__ CUtensorMap tm64, const TileParams p) {
  using Cfg = TileCfg<NT, SPLIT>;
  constexpr int kW = Cfg::kW, kB = Cfg::kB, kDBufs = Cfg::kDBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* wfull = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBar);
  uint64_t* wempty = wfull + kW;
  uint64_t* bfull = wempty + kW;
  uint64_t* bempty = bfull + kB;
  uint64_t* afull = bempty + kB;
  uint64_t* aempty = afull + kABufs;
  uint64_t* dfull = aempty + kABufs;
  uint64_t* dempty = dfull + kDBufs;
  uint64_t* mma_done = dempty + kDBufs;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 4);
  int* s_total = reinterpret_cast<int*>(smem + Cfg::kOffMisc + 8);
  int* s_prefix = reinterpret_cast<int*>(smem + Cfg::kOffPrefix);
  int* s_offs = reinterpret_cast<int*>(smem + Cfg::kOffOffs);
  const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t sbase = uniform(smem_u32(smem));
  const uint32_t b_wfull = sbase + Cfg::kOffBar, b_wempty = b_wfull + 8 * kW;
  const uint32_t b_bfull = b_wempty + 8 * kW, b_bempty = b_bfull + 8 * kB;
  const uint32_t b_afull = b_bempty + 8 * kB, b_aempty = b_afull + 8 * kABufs;
  const uint32_t b_dfull = b_aempty + 8 * kABufs, b_dempty = b_dfull + 8 * kDBufs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kW; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], kExpandWarps / 2);
    }
    for (int s = 0; s < kB; ++s) {
      mbar_init(&bfull[s], GATHER ? kGatherThreads : 1);
      mbar_init(&bempty[s], 2);
    }
    for (int i = 0; i < kABufs; ++i) {
      mbar_init(&afull[i], kExpandWarps / 2);
      mbar_init(&aempty[i], 2);
    }
    for (int i = 0; i < kDBufs; ++i) {
      mbar_init(&dfull[i], 2);
      mbar_init(&dempty[i], 4);
    }
    mbar_init(mma_done, 2);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == kTokenWarp && lane == 0 && !GATHER) {
    tma_prefetch_desc(&tm16);
    tma_prefetch_desc(&tm64);
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  // `early`: the offsets were written before the launch that this one follows, so
  // weights may stream at once and only the token rows have to be waited for
  if (!p.early) pdl_wait_and_trigger();
  if (warp == 2)
    build_tile_table<NT>(p.offsets, p.n_groups, p.dense_rows, p.out_rows, s_prefix, s_offs, s_total,
                         p.status, lane);
  tc_fence_before();
  if constexpr (SPLIT)
    cluster_sync_all();        // also: the peers run, so their shared memory may be written
  else
    __syncthreads();
  tc_fence_after();
  // All columns are this CTA's, so they start at 0; as a constant, that makes the MMAs'
  // operands uniform.
  if (*s_tmem != 0u && threadIdx.x == 0) report(p.status, MOE_ERR_CUDA);
  const int total = static_cast<int>(uniform(*s_tmem == 0u ? static_cast<uint32_t>(*s_total * p.blocks) : 0u));
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = SPLIT ? static_cast<int>(blockIdx.x) / p.splits : static_cast<int>(blockIdx.x);
  const int step = SPLIT ? total : static_cast<int>(gridDim.x);   // a cluster has one item
  // records of this CTA; a half of the last one may be past K: zero weights, zero tokens
  const int kb0 = SPLIT ? p.kb * rank / p.splits : 0;
  const int kb1 = SPLIT ? p.kb * (rank + 1) / p.splits : p.kb;
  // item w: chunk w / blocks; tiles of row block w % blocks
  // The items of the last round go to twice as many CTAs, a tile each, where these are
  // idle otherwise (K 7168, N 4096: 16384 tokens 557 us, 569; 1536 tokens 75, 82).  With an odd
  // number of row tiles the last block's second item has none: its CTA loads tokens only.
  const int rest = GATHER || SPLIT || p.swiglu ? 0 : total % static_cast<int>(gridDim.x);
  const int whole = total - (2 * rest <= static_cast<int>(gridDim.x) ? rest : 0);
  const int count = 2 * total - whole;
  auto chunk_of = [&](int w) { return w < whole ? w : whole + (w - whole) / 2; };
  auto first_tile = [&](int w) { return w < whole ? 0 : (w - whole) & 1; };
  auto tiles_of = [&](int w, int b) {
    return p.swiglu ? 2 : max(0, min(w < whole ? 2 : 1, p.rt - 2 * b - first_tile(w)));
  };

  if (warp == 0) {
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 0, parity = 0, issued = 0;
      bool ok = true;
      for (int w = first; w < count && ok; w += step) {
        const Tile t = decode_tile<NT>(chunk_of(w), p.blocks, p.n_groups, s_prefix, s_offs);
        const int nt = tiles_of(w, t.nt);
        const uint8_t* src = p.w + p.matrix * (static_cast<size_t>(t.g) * (p.swiglu ? 2 : 1)) +
                             (static_cast<size_t>(p.swiglu ? t.nt : 2 * t.nt + first_tile(w)) * p.kb + kb0) * p.record;
        const size_t next = p.swiglu ? p.matrix : static_cast<size_t>(p.kb) * p.record;
        for (int kb = kb0; kb < kb1; ++kb, src += p.record) {
          if (!mbar_wait(&wempty[slot], phase ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          mbar_expect_tx(&wfull[slot], p.record * nt);
          for (int i = 0; i < nt; ++i)
            bulk_load(smem + Cfg::kOffW + slot * kWStage + i * kMaxRecord, src + next * i, p.record,
                      &wfull[slot]);
          issued |= 1u << slot;
          parity = (parity & ~(1u << slot)) | (phase << slot);
          advance(slot, phase, kW);
        }
      }
      if (!ok) fail(s_abort, p.status);
      // nothing may be in flight into this shared memory when the CTA ends
      for (int s = 0; s < kW; ++s)
        if ((issued >> s) & 1u) mbar_wait(&wfull[s], (parity >> s) & 1u, nullptr);
    }
    __syncwarp();
  } else if (warp == 1 || warp == kMmaWarp) {
    if (p.early) pdl_wait_and_trigger();
    const uint32_t tile = warp == 1 ? 0u : 1u;
    int bs = 0, ab = 0, db = 0;
    uint32_t bphase = 0, aphase = 0, dphase = 0;
    bool ok = true;
    for (int w = first; w < count && ok; w += step) {
      const Tile t = decode_tile<NT>(chunk_of(w), p.blocks, p.n_groups, s_prefix, s_offs);
      const bool mine = uniform(tile < tiles_of(w, t.nt)) != 0u;
      const uint32_t idesc = uniform(idesc_bf16_f32(128, (t.rows + 15) / 16 * 16));
      const uint32_t d = kTmemD + static_cast<uint32_t>(db * 2 + tile) * NT;
      ok = warp_wait(b_dempty + 8 * db, dphase ^ 1u, s_abort);
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        // both in one vote, as a wait on a barrier that is ready costs 100 clocks and more
        const bool both = __all_sync(0xffffffffu, try_wait_at(b_bfull + 8 * bs, bphase) &
                                                      try_wait_at(b_afull + 8 * ab, aphase));
        ok = both || (warp_wait(b_bfull + 8 * bs, bphase, s_abort) && warp_wait(b_afull + 8 * ab, aphase, s_abort));
        if (!ok) break;
        if (mine) {
          tc_fence_after();
          const uint64_t b = sdesc_sw128(sbase + static_cast<uint32_t>(bs) * Cfg::kTok);
          const uint32_t a = static_cast<uint32_t>(ab) * kACols + tile * (kACols / 2);
          umma_bf16_ts64(d, a, b, idesc, kb != kb0);
          umma_bf16_ts64(d, a + 32, b + (NT * 128 >> 4), idesc, 1u);
        }
        commit_at(b_aempty + 8 * ab);
        advance(ab, aphase, kABufs);
        commit_at(b_bempty + 8 * bs);
        advance(bs, bphase, kB);
      }
      if (!ok) break;
      commit_at(b_dfull + 8 * db);
      advance(db, dphase, kDBufs);
    }
    if (!ok && lane == 0) fail(s_abort, p.status);
    commit_at(smem_u32(mma_done));
    mbar_wait(mma_done, 0u, nullptr);
    __syncwarp();
  } else if (warp >= 6 && warp < kMmaWarp) {
    if (p.early) pdl_wait_and_trigger();
    const int set = (warp - 6) >> 3, tile = ((warp - 6) >> 2) & 1, r = (warp & 3) * 32 + lane;
    const uint32_t d = (static_cast<uint32_t>((warp & 3) * 32) << 16) +
                       static_cast<uint32_t>(set * kACols + tile * (kACols / 2));
    const uint32_t swap = static_cast<uint32_t>((r >> 1) & 3) << 4;
    const uint32_t codes = sbase + Cfg::kOffW + tile * kMaxRecord + r * 64;
    const uint32_t scales = sbase + Cfg::kOffW + tile * kMaxRecord + kQCodeBytes +
                            r * (p.group == 16 ? 8 : 4);
    int slot = set, n = 0;                        // n: records before this item
    uint32_t phase = 0, aphase = 1;
    bool ok = true;
    for (int w = first; w < count && ok; w += step) {
      const bool mine = uniform(tile < tiles_of(w, chunk_of(w) % p.blocks)) != 0u;
      for (int kb = kb0 + ((n ^ set) & 1); kb < kb1; kb += 2) {
        ok = warp_wait(b_wfull + 8 * slot, phase, s_abort);
        if (!ok) break;
        uint4 c[4];                               // pieces
        uint2 sc = make_uint2(0u, 0u);
        if (mine) {
          const uint32_t at = codes + slot * kWStage;
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) c[i] = lds128(at + ((i << 4) ^ swap));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc.x) : "r"(scales + slot * kWStage) : "memory");
          if (p.group == 16)
            asm volatile("ld.shared.b32 %0, [%1+4];" : "=r"(sc.y) : "r"(scales + slot * kWStage) : "memory");
          else           // a byte for every 32 inputs, twice
            sc = make_uint2(__byte_perm(sc.x, 0u, 0x1100), __byte_perm(sc.x, 0u, 0x3322));
        }
        __syncwarp();
        if (lane == 0) arrive_at(b_wempty + 8 * slot);
        slot += 2;
        if (slot >= kW) {
          slot -= kW;
          phase ^= 1u;
        }
        ok = warp_wait(b_aempty + 8 * set, aphase, s_abort);
        if (!ok) break;
        if (mine) {
          tc_fence_after();
          if (p.code == MOE_QUANT_INT) {
            expand_half<MOE_QUANT_INT>(c[0], c[1], sc.x, d);
            expand_half<MOE_QUANT_INT>(c[2], c[3], sc.y, d + 32);
          } else {
            expand_half<MOE_QUANT_E2M1>(c[0], c[1], sc.x, d);
            expand_half<MOE_QUANT_E2M1>(c[2], c[3], sc.y, d + 32);
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(b_afull + 8 * set);
        aphase ^= 1u;
      }
      n += kb1 - kb0;
    }
    if (!ok && lane == 0) fail(s_abort, p.status);
  } else if (!GATHER && warp == kTokenWarp) {
    if (p.early) pdl_wait_and_trigger();
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 0, parity = 0, issued = 0;
      bool ok = true;
      for (int w = first; w < count && ok; w += step) {
        const Tile t = decode_tile<NT>(chunk_of(w), p.blocks, p.n_groups, s_prefix, s_offs);
        const int nb = (t.rows + 15) / 16;
        const bool wide = nb > 2;
        const int boxes = wide ? (t.rows + 63) / 64 : nb, box = wide ? 64 : 16;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&bempty[slot], phase ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          mbar_expect_tx(&bfull[slot], static_cast<uint32_t>(2 * boxes * box * kHalf * 2));
          for (int j = 0; j < 2; ++j)
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(smem + slot * Cfg::kTok + j * (NT * 128) + i * box * kHalf * 2,
                          wide ? &tm64 : &tm16, &bfull[slot], kb * kQK + j * kHalf,
                          t.row0 + i * box);
          issued |= 1u << slot;
          parity = (parity & ~(1u << slot)) | (phase << slot);
          advance(slot, phase, kB);
        }
      }
      if (!ok) fail(s_abort, p.status);
      for (int s = 0; s < kB; ++s)
        if ((issued >> s) & 1u) mbar_wait(&bfull[s], (parity >> s) & 1u, nullptr);
    }
    __syncwarp();
  } else if (GATHER && warp >= kTokenWarp) {
    // Thread g copies the 16-byte piece g % 8 of token rows g / 8 + 16 i of a stage; a
    // piece lands at piece ^ (row % 8) of its 128-byte row.  Pieces past K are zero
    // (their weights are, but zero times NaN is not), and so is a token out of range.
    // A stage's copies are one cp.async group, reported kLag groups later (8192 tokens of 128
    // experts 593 us, 600 with a lag of 2).
    constexpr int kLag = 1, kPer = NT / 16;
    const int g = threadIdx.x - kTokenWarp * 32, piece = g & 7, rg = g >> 3;
    int slot = 0, aslot = 0, pending = 0;
    uint32_t phase = 0;
    bool ok = true, bad = false;
    // an item's tokens are loaded while the rows of the one before it are copied
    Tile t{};
    int tok[kPer];
    auto look = [&](int w) {
      t = decode_tile<NT>(chunk_of(w), p.blocks, p.n_groups, s_prefix, s_offs);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        tok[i] = rg + 16 * i < t.rows ? __ldg(p.token + t.row0 + rg + 16 * i) : 0;
    };
    if (first < count) look(first);
    for (int w = first; w < count && ok; w += step) {
      const int rows = t.rows;
      const uint4* src[kPer];
      uint32_t size[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool fine = tok[i] >= 0 && tok[i] < p.x_rows;
        bad |= !fine;
        src[i] = p.x + static_cast<size_t>(fine ? tok[i] : 0) * (p.ldx / 8) + kb0 * (kQK / 8) + piece;
        size[i] = fine ? 16u : 0u;
      }
      if (w + step < count) look(w + step);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!try_wait_at(b_bempty + 8 * slot, phase ^ 1u) &&
            !wait_on(b_bempty + 8 * slot, phase ^ 1u, s_abort)) {
          ok = false;
          break;
        }
        const uint32_t sb = sbase + slot * Cfg::kTok + rg * 128 + ((piece ^ (rg & 7)) << 4);
        const int k = kb * kQK + piece * 8;
        const uint32_t in0 = k < p.K ? 16u : 0u, in1 = k + kHalf < p.K ? 16u : 0u;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (16 * i >= rows) break;
          if (rg + 16 * i < rows) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sb + i * 16 * 128),
                         "l"(src[i]), "r"(size[i] & in0)
                         : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sb + NT * 128 + i * 16 * 128),
                         "l"(src[i] + kHalf / 8), "r"(size[i] & in1)
                         : "memory");
          }
          src[i] += kQK / 8;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++pending > kLag) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
          fence_proxy_async_smem();
          mbar_arrive(&bfull[aslot]);
          if (++aslot == kB) aslot = 0;
          --pending;
        }
        advance(slot, phase, kB);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    if (ok) {
      for (; pending > 0; --pending) {
        mbar_arrive(&bfull[aslot]);
        if (++aslot == kB) aslot = 0;
      }
    } else if (lane == 0) {
      fail(s_abort, p.status);
    }
    if (bad) report(p.status, MOE_ERR_BAD_INDEX);
  } else if (warp >= 2 && warp < 6) {
    if (p.early) pdl_wait_and_trigger();
    const int q = warp & 3, r = q * 32 + lane;
    int db = 0;
    uint32_t dphase = 0;
    bool ok = true;
    for (int w = first; w < count; w += step) {
      const Tile t = decode_tile<NT>(chunk_of(w), p.blocks, p.n_groups, s_prefix, s_offs);
      const int nt = tiles_of(w, t.nt);
      const float u = p.code == MOE_QUANT_E2M1 ? quant_unit<MOE_QUANT_E2M1>() : quant_unit<MOE_QUANT_INT>();
      const float f0 = __ldg(p.factor + (p.swiglu ? 2 * t.g : t.g)) * u;
      const float f1 = p.swiglu ? __ldg(p.factor + 2 * t.g + 1) * u : f0;
      ok = warp_wait(b_dfull + 8 * db, dphase, s_abort);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = kTmemD + (static_cast<uint32_t>(q * 32) << 16) +
                         static_cast<uint32_t>(db * 2 * NT);
      if constexpr (SPLIT) {
        // A CTA sums `per` of the chunk's columns: its slot [rank][per / 2][256 rows] of
        // pairs
        const uint32_t part = sbase + Cfg::kOffPart;
        const int per = columns_of(t.rows, p.splits);
        for (int i = 0; i < nt; ++i)
          for (int c0 = 0; c0 < t.rows; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(d + static_cast<uint32_t>(i * NT + c0), v);
            tmem_ld_wait();
            const float f = i == 0 ? f0 : f1;
#pragma unroll
            for (int c = 0; c < 16; c += 2) {     // pairs: per is even
              const int to = (c0 + c) / per, in = c0 + c - to * per;
              asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                               mapa_shared(part, static_cast<uint32_t>(to)) +
                               static_cast<uint32_t>(((rank * (per / 2) + in / 2) * 256 + i * 128 + r) * 8)),
                           "f"(__uint_as_float(v[c]) * f), "f"(__uint_as_float(v[c + 1]) * f)
                           : "memory");
            }
          }
      } else if (p.f32) {
        for (int i = 0; i < nt; ++i) {
          const int col = (2 * t.nt + first_tile(w) + i) * 128 + r;
          float* out = static_cast<float*>(p.out) + static_cast<size_t>(t.row0) * p.ldo + col;
          for (int c0 = 0; c0 < t.rows; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(d + static_cast<uint32_t>(i * NT + c0), v);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c, out += p.ldo)
              if (c0 + c < t.rows && col < p.n) *out = __uint_as_float(v[c]) * f0;
          }
        }
      } else {
        // 32 features of 16 tokens at a time: as bf16 through shared memory, where a token
        // has its features in a row, in 16-byte pieces (octets of features) to memory
        const uint32_t stage = sbase + Cfg::kOffOut + q * 1024;
        const uint32_t put = stage + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
        const uint32_t get = stage + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
        const int outs = p.swiglu ? 1 : nt;
        for (int i = 0; i < outs; ++i) {
          const int col = (p.swiglu ? t.nt : 2 * t.nt + first_tile(w) + i) * 128 + q * 32 + (lane & 3) * 8;
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) +
                               static_cast<size_t>(t.row0 + (lane >> 2)) * p.ldo + col;
          const bool whole = p.vec && col + 8 <= p.n;
          for (int c0 = 0; c0 < t.rows; c0 += 16) {
            float v[2][8];                        // [lanes 0-15, 16-31]
            tmem_ld_frag(d + static_cast<uint32_t>(i * NT + c0), v[0]);
            tmem_ld_frag(d + (16u << 16) + static_cast<uint32_t>(i * NT + c0), v[1]);
            // Activations leave as one bf16, as the bf16 layer's do, though the next product
            // sums them in fp32: a second bf16 with what is left would double that product's
            // MMAs and token rows, which bound it for many tokens.  The error of the outputs
            // is 0.0023 so, their own rounding's 0.0016 without.
            if (p.swiglu) {
              float up[2][8];
              tmem_ld_frag(d + static_cast<uint32_t>(NT + c0), up[0]);
              tmem_ld_frag(d + (16u << 16) + static_cast<uint32_t>(NT + c0), up[1]);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                v[j / 8][j % 8] = silu_fast(v[j / 8][j % 8] * f0) * (up[j / 8][j % 8] * f1);
            } else {
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j / 8][j % 8] *= f0;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {         // eight tokens each
              const uint32_t m[4] = {pack_bf16x2(v[0][4 * b], v[0][4 * b + 1]),
                                     pack_bf16x2(v[0][4 * b + 2], v[0][4 * b + 3]),
                                     pack_bf16x2(v[1][4 * b], v[1][4 * b + 1]),
                                     pack_bf16x2(v[1][4 * b + 2], v[1][4 * b + 3])};
              __syncwarp();                       // this buffer's last tokens have been read
              stmatrix_trans(put + b * 512, m);
              __syncwarp();
              const uint4 o = lds128(get + b * 512);
              const int left = t.rows - c0 - 8 * b - (lane >> 2);
              if (left > 0) {
                if (whole) {
                  *reinterpret_cast<uint4*>(out) = o;
                } else {
                  const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    if (col + j < p.n)
                      out[j] = __ushort_as_bfloat16(static_cast<unsigned short>(w[j / 2] >> (16 * (j & 1))));
                }
              }
              out += 8 * p.ldo;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&dempty[db]);
      advance(db, dphase, kDBufs);
    }
    if (!ok && lane == 0) fail(s_abort, p.status);
  }

  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();          // every partial sum has arrived
    if (first < total && *s_abort == 0) {
      const Tile t = decode_tile<NT>(first, p.blocks, p.n_groups, s_prefix, s_offs);
      const float2* part = reinterpret_cast<const float2*>(smem + Cfg::kOffPart);
      const int per = columns_of(t.rows, p.splits);
      const int rows = p.swiglu ? 128 : 256;
      // neighbouring threads: neighbouring features
      for (int i = threadIdx.x; i < per / 2 * rows; i += blockDim.x) {
        const int c = i / rows * 2, r = i % rows;
        const int col = t.nt * rows + r;
        float2 y = make_float2(0.f, 0.f), v = y;
        for (int s = 0; s < p.splits; ++s) {
          const float2 a = part[(s * (per / 2) + c / 2) * 256 + r];
          y.x += a.x;
          y.y += a.y;
          if (p.swiglu) {
            const float2 b = part[(s * (per / 2) + c / 2) * 256 + 128 + r];
            v.x += b.x;
            v.y += b.y;
          }
        }
        if (p.swiglu) y = make_float2(silu_fast(y.x) * v.x, silu_fast(y.y) * v.y);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int token = rank * per + c + k;
          if (token >= t.rows || col >= p.n) continue;
          const size_t at = static_cast<size_t>(t.row0 + token) * p.ldo + col;
          if (p.f32)
            static_cast<float*>(p.out)[at] = k == 0 ? y.x : y.y;
          else
            static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(k == 0 ? y.x : y.y);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(*s_tmem, 512);
  }
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

template <int NT, bool GATHER, bool SPLIT>
cudaError_t launch_tile(const CUtensorMap& tm16, const CUtensorMap& tm64, const TileParams& p,
                        unsigned grid, cudaStream_t s) {
  using Cfg = TileCfg<NT, SPLIT>;
  static bool done[64] = {false};
  auto kern = quant_tile_kernel<NT, GATHER, SPLIT>;
  const cudaError_t e = set_smem_once(kern, static_cast<int>(Cfg::kSmem), done);
  if (e != cudaSuccess) return e;
  const dim3 block(GATHER ? kThreadsGather : kThreads);
  if (!SPLIT) return launch_pdl(kern, dim3(grid), block, Cfg::kSmem, s, tm16, tm64, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tm16, tm64, p);
}

// Clusters of `size` CTAs of the splitting kernel that the device holds at once.
int clusters_at_once(int size) {
  static int cache[64][kMaxSplits + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int& n = cache[dev][size];
  if (n == 0) {
    using Cfg = TileCfg<64, true>;
    auto kern = quant_tile_kernel<64, false, true>;
    static bool done[64] = {false};
    if (set_smem_once(kern, static_cast<int>(Cfg::kSmem), done) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
    (void)cudaGetLastError();
  }
  return n;
}

}  // namespace

cudaError_t launch_quant_gemm(const QuantGemmArgs& a, cudaStream_t s) {
  TileParams p{};
  const QuantShape q = quant_shape(a.n, a.K, a.group);
  p.w = static_cast<const uint8_t*>(a.w);
  p.factor = reinterpret_cast<const float*>(p.w + q.bytes * a.n_groups * (a.swiglu ? 2 : 1));
  p.x = static_cast<const uint4*>(a.x);
  p.token = a.token;
  p.offsets = a.offsets;
  p.out = a.out;
  p.ldx = a.ldx;
  p.ldo = a.ldo;
  p.out_rows = a.out_rows;
  p.matrix = q.bytes;
  p.record = quant_record(a.group);
  p.n_groups = a.n_groups;
  p.dense_rows = a.dense_rows;
  p.x_rows = a.x_rows;
  p.n = a.n;
  p.K = a.K;
  p.kb = q.kb;
  p.rt = q.rt;
  p.blocks = a.swiglu ? q.rt : (q.rt + 1) / 2;
  p.code = a.code;
  p.group = a.group;
  p.swiglu = a.swiglu != 0;
  p.f32 = a.out_f32;
  p.vec = a.ldo % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0;
  p.early = a.early && a.token == nullptr;
  p.splits = 1;
  p.status = a.status;
  CUtensorMap tm16{}, tm64{};
  if (a.token == nullptr) {
    const bool ok = a.ldx == a.K ? make_tmap_bf16(&tm16, a.x, a.x_rows, a.K, 16) &&
                                       make_tmap_bf16(&tm64, a.x, a.x_rows, a.K, 64)
                                 : encode_tmap(&tm16, a.x, 2, a.x_rows, a.K, a.ldx, 16, 64) &&
                                       encode_tmap(&tm64, a.x, 2, a.x_rows, a.K, a.ldx, 64, 64);
    if (!ok) return cudaErrorInvalidValue;
  }
  // chunks of nt tokens that there can be, as every group may end inside one
  auto items_of = [&](int nt) {
    const long long chunks = a.offsets == nullptr ? (a.dense_rows + nt - 1) / nt
                                                  : a.out_rows / nt + std::min(a.out_rows, static_cast<long long>(a.n_groups));
    return chunks * p.blocks;
  };
  // Chunks of 128 tokens where the groups' mean passes 64, as a weight is expanded for a
  // chunk (8192 tokens of 128 experts 581 us, 709 in chunks of 64; 16384 tokens of K 7168, N 4096
  // 557, 856; but 900 tokens of the experts, 56 a group, 122 in 64, 130 in 128), nor where chunks
  // of 64 are at most an item an SM: there an item's length counts (512 tokens of K 7168,
  // N 4096 36 us, in chunks of 128 41; 333 tokens of 12 experts 12.4, 16.3).
  const bool wide = a.out_rows > 64ll * a.n_groups && items_of(64) > a.sm_count;
  const long long items = items_of(wide ? 128 : 64);
  if (a.token == nullptr && a.offsets == nullptr && !wide) {
    // A cluster's CTAs split K where whole items leave SMs idle, as wide as clusters fit at
    // once (64, 128 and 256 tokens of K 7168, N 4096 12.5, 15.5 and 23.3 us, an item a CTA 35;
    // 152 SMs hold 15 clusters of eight, so 64 tokens took 22 us in 16 of eight, 14.6 in
    // clusters of four, 13 in six).
    int splits = kMaxSplits;
    while (splits > 1 && (items > clusters_at_once(splits) || p.kb < splits)) --splits;
    if (splits > 1) {
      p.splits = splits;
      return launch_tile<64, false, true>(tm16, tm64, p, static_cast<unsigned>(items * splits), s);
    }
  }
  const unsigned grid = static_cast<unsigned>(std::min(items, static_cast<long long>(a.sm_count)));
  if (a.token != nullptr)
    return wide ? launch_tile<128, true, false>(tm16, tm64, p, grid, s)
                : launch_tile<64, true, false>(tm16, tm64, p, grid, s);
  return wide ? launch_tile<128, false, false>(tm16, tm64, p, grid, s)
              : launch_tile<64, false, false>(tm16, tm64, p, grid, s);
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
