// tc.cuh -- a persistent matrix product on the 5th-generation tensor cores:
// TMA-fed shared-memory ring, tcgen05.mma into TMEM, and an epilogue functor
// that gets the float32 accumulator 32 columns at a time.
//
//   C(m, n) = sum over terms (pa, pb), sum over k of A[pa](m, k) * B[pb](n, k)
//
// A and B are bfloat16 with float32 accumulation.  float32 operands come as
// three bfloat16 planes whose sum is the value to 24 bits (hi, mid, lo, each
// the rounding of what the ones before left over); the six products of planes
// down to 2^-16 of the first are then the `terms`, smallest first so that the
// accumulator's rounding acts on small values while it is small.
//
// Either operand may be K-major (k contiguous in memory) or MN-major (m or n
// contiguous): the shared-memory descriptors and the instruction descriptor
// say which, so no operand is ever transposed in memory.
//
// Two CTAs (a cluster, one an SM) work on one 256 x 256 tile: each loads its
// 128 rows of A and half of B's 256 rows, so a stage brings 64 KB for 256 x
// 256 x 64 products instead of the 96 KB of two 128 x 256 tiles -- per SM 64
// bytes a cycle at the tensor cores' full rate --, and the first CTA's
// tcgen05.mma reads both CTAs' shared memory and writes both CTAs' TMEM.  In
// each CTA warps 0-7 run the epilogue of its 128 rows (warp w reads TMEM lanes
// 32 (w % 4) .. + 31 and column half w / 4), warp 8 issues the copies; warp 9
// of the first CTA issues the matrix instructions.  The accumulator is
// double-buffered in TMEM (2 x 256 columns), so an epilogue runs under the
// next product.
//
// The accumulator of a tensor core drops bits where IEEE addition would
// round (measured: the error of a sum grows with its number of k steps,
// 1.7e-6 of a log-probability at k = 4096 against 3e-7 in plain float32; a sum
// of one sign loses about 2e-7 of itself at each step of 16 k).
// A new accumulator therefore starts every GROUP stages, and the partial sums
// are added in float32 registers; the TMEM reads cost 7% of the time at 8
// stages, 2 to 3% at 16.  GROUP = 0 is for sums that are no longer than a group
// anyway: their epilogue works on the accumulator straight from TMEM, with
// fewer registers.
//
// Every wait is bounded: a wait that gives up records the timeout in the
// status word and raises a shared flag that ends the CTA's roles (the other
// CTA's waits then run out too).  Each wait covers a few stages or one
// accumulator, never the product, so its limit holds for products of any
// length.  Once the roles of both CTAs have ended, copies and matrix
// instructions in flight are waited for (bounded) before TMEM is freed and the
// cluster ends together.
#pragma once

#include <type_traits>

#include "tma.cuh"

namespace rlca {

constexpr int kTcM = 256;      // rows of a tile, half of them each CTA's
constexpr int kTcN = 256;      // columns of a tile; each CTA copies half of B's rows
constexpr int kTcK = 64;       // k per stage: one 128-byte swizzle row of bfloat16
constexpr int kTcStages = 6;
constexpr int kTcRows = kTcM / 2;  // rows a CTA loads and finishes
constexpr int kTcEpiWarps = 8;
constexpr int kTcThreads = 32 * (kTcEpiWarps + 4);  // two warps idle: register shares go by four warps
// registers a thread: 168 at launch (384 threads), then 208 for the epilogue's
// 256 threads and 88 for the other 128 -- the same 64,512 in all
constexpr int kTcEpiRegs = 208, kTcIssueRegs = 88;
static_assert(32 * (kTcEpiWarps * kTcEpiRegs + 4 * kTcIssueRegs) <= 168 * kTcThreads, "shares within the launch's registers");
constexpr int kTcABytes = kTcRows * kTcK * 2;
constexpr int kTcBBytes = kTcN / 2 * kTcK * 2;
constexpr int kTcStageBytes = kTcABytes + kTcBBytes;
constexpr size_t kTcSmem = (size_t)kTcStages * kTcStageBytes + 1024;  // + alignment of the ring
// ... and, where an epilogue asks for them, a 32 x 32 block of each of its
// warps, rows padded against bank conflicts (otherwise L1 keeps the 33 KB)
constexpr int kTcBlockFloats = 32 * 33;
constexpr size_t kTcSmemBlocks = kTcSmem + kTcEpiWarps * kTcBlockFloats * 4;
static_assert(kTcSmemBlocks + 512 <= 227 * 1024, "with the barriers, within a CTA's shared memory");

// the plane pairs of one product, four bits each for A's and B's plane
struct TcTerms {
  int n;
  unsigned char a[6], b[6];
};

struct TcShape {
  // extents; the one named by `count_axis` is *count, known on the device only
  const int* count;
  int count_axis;  // 0: none, 1: m, 2: k
  int m, n, k;
  // added to the tensor maps' coordinates: A's m, B's n, B's k
  int a_m0, b_n0, b_k0;
  int splits;      // the k axis in this many parts (each its own output)
  int band;        // row tiles walked together before the next column tile
  // where *count == full, map_other stands for A's (other = 1) or B's (2)
  int other, full;
  TcTerms terms;
};

// ---- tcgen05 ------------------------------------------------------------------
__device__ __forceinline__ void tc_alloc(uint32_t* smem_dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// arrives on `bar` -- of both CTAs -- once every matrix instruction issued so
// far has completed
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Starts the load of 32 columns of this warp's 32 TMEM lanes (one row a
// thread); the values are there after tc_load_wait.
__device__ __forceinline__ void tc_load32(uint32_t addr, float (&v)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr)
      : "memory");
}
// waits for this thread's loads so far; v passes through so that its uses stay behind the wait
__device__ __forceinline__ void tc_load_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[i]));
}

// ... 16 columns, added to v
__device__ __forceinline__ void tc_add16(uint32_t addr, float* v) {
  uint32_t r[16];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  // (the registers pass through behind the wait, so that their uses stay behind it too)
#pragma unroll
  for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(r[i]);
}

// Shared-memory matrix descriptor of a 128-byte-swizzled tile at `addr`
// (1024-byte aligned but for the k offset inside a swizzle row).  K-major:
// rows of 128 bytes, groups of 8 rows 1024 bytes apart.  MN-major: blocks of
// 64 values of m (or n) x kTcK values of k, a block's 8-k groups 1024 bytes
// apart, blocks kTcK * 128 bytes apart.
template <bool MN>
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr) {
  const uint64_t lead = MN ? (kTcK * 128) >> 4 : 1, stride = 1024 >> 4;
  return (uint64_t)((addr & 0x3ffff) >> 4) | (lead << 16) | (stride << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// ... advanced by 16 values of k
template <bool MN>
constexpr uint64_t kTcStepK = MN ? (2 * 1024) >> 4 : 32 >> 4;

// bfloat16 x bfloat16 -> float32, M = 256, N = 256
template <bool A_MN, bool B_MN>
constexpr uint32_t kTcInstr = (1u << 4) | (1u << 7) | (1u << 10) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) |
                              ((uint32_t)(kTcN >> 3) << 17) | ((uint32_t)(kTcM >> 4) << 24);

// ---- registers of a warpgroup (all its warps together) -------------------------
template <int N>
__device__ __forceinline__ void regs_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- the two CTAs of a cluster -----------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// cluster-wide address of the first CTA's copy of a shared variable
__device__ __forceinline__ uint32_t in_first(const void* p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
// (what the arrival hands over is TMEM, ordered by the tcgen05 fences; a
// release at cluster scope would wait for the epilogue's stores to memory)
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// a copy into this CTA's shared memory, counted by the barrier at `bar`
// (which may be the other CTA's)
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// a bounded wait that also ends when another role has given up
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* stop) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*stop) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      atomicOr(&g_tu_status, kStatusWaitTimeout);
      *stop = 1;
      return false;
    }
  }
}

// ---- tiles ------------------------------------------------------------------------
struct TcTile {
  int m0, n0, split, k_begin, k_end;  // k in stages
};

struct TcWalk {
  int count, m, k, mt, nt, k_stages, per_split;
  int64_t tiles;
  __device__ TcWalk(const TcShape& s) {
    count = s.count ? *s.count : 0;
    m = s.count_axis == 1 ? min(count, s.m) : s.m;
    k = s.count_axis == 2 ? min(count, s.k) : s.k;
    mt = (m + kTcM - 1) / kTcM;
    nt = (s.n + kTcN - 1) / kTcN;
    k_stages = (k + kTcK - 1) / kTcK;
    per_split = (k_stages + s.splits - 1) / s.splits;
    tiles = (int64_t)mt * nt * s.splits;
  }
  // bands of row tiles; inside a band the row tile runs fastest, so CTAs that
  // run together share the band's rows of A and a few column tiles of B
  __device__ TcTile at(int64_t t, const TcShape& s) const {
    const int64_t plane = (int64_t)mt * nt;
    TcTile r;
    r.split = (int)(t / plane);
    t -= r.split * plane;
    const int64_t per_band = (int64_t)s.band * nt;
    const int band = (int)(t / per_band);
    t -= band * per_band;
    const int rows = min(s.band, mt - band * s.band);
    r.n0 = (int)(t / rows) * kTcN;
    r.m0 = (band * s.band + (int)(t % rows)) * kTcM;
    r.k_begin = min(k_stages, r.split * per_split);
    r.k_end = min(k_stages, r.k_begin + per_split);
    return r;
  }
};

// End of the accumulation that starts at step `at` of terms x stages steps.
// All terms but the last are at most 2^-8 of it: they share accumulators of
// kTcLead steps, whose dropped bits are that much smaller.  (An accumulator
// bounds the epilogue's wait, too: the lead terms of 16 million rows in one
// would be 0.35 s, longer than a wait may last.)
constexpr int kTcLead = 128;  // about 35 us
template <int GROUP>
__host__ __device__ constexpr int tc_group_end(int at, int stages, int terms) {
  const int all = stages * terms, lead = stages * (terms - 1);
  static_assert(GROUP <= kTcLead);
  if (GROUP == 0) return all;
  const int end = at < lead ? at + kTcLead : at + GROUP, last = at < lead ? lead : all;
  return end < last ? end : last;
}

// One product.  Epi: struct State; begin(State&, walk, tile, row, col0) with
// row = the thread's row of C and col0 the first column of its half tile;
// chunk(State&, col, v[32], block) for the 32 columns from col on, by whole
// warps, with a shared-memory block of the warp's own (if the launch has
// kTcSmemBlocks); end(State&).  Rows from
// walk.m on do not exist.
template <bool A_MN_, bool B_MN_, int GROUP_, class Epi_>
struct TcJob {
  using Epi = Epi_;
  static constexpr bool A_MN = A_MN_, B_MN = B_MN_;
  static constexpr int GROUP = GROUP_;
  CUtensorMap a, b, other;
  TcShape s;
  Epi epi;
};
struct TcNoJob {
  static constexpr int GROUP = 0;
};
// whether the epilogue's partial sums take registers from the other warps
template <class Job1, class Job2>
constexpr bool kTcShares = Job1::GROUP > 0 || Job2::GROUP > 0;

// what a CTA's roles share
struct TcShared {
  // of the first CTA: full, acc_empty; of both: empty, acc_full, drained
  uint64_t full[kTcStages], empty[kTcStages], acc_full[2], acc_empty[2], drained;
  uint32_t tmem_base;
  volatile int stop;
};

// the ring of stages as a role sees it
struct TcRing {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kTcStages) stage = 0, phase ^= 1;
  }
};
// ... and the two accumulators
struct TcAcc {
  int buf = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    buf ^= 1;
    if (buf == 0) phase ^= 1;
  }
};

// Copies of one tile; false once a wait has given up.
template <class Job>
__device__ __forceinline__ bool tc_copy_tile(const Job& job, const TcWalk& walk, int64_t t, int rank, TcShared& sh,
                                             unsigned char* ring, TcRing& r) {
  const TcShape& s = job.s;
  const bool other = s.other != 0 && walk.count == s.full;
  const CUtensorMap* ma = other && s.other == 1 ? &job.other : &job.a;
  const CUtensorMap* mb = other && s.other == 2 ? &job.other : &job.b;
  const TcTile tile = walk.at(t, s);
  const int m0 = s.a_m0 + tile.m0 + rank * kTcRows, n0 = s.b_n0 + tile.n0 + rank * (kTcN / 2);
  for (int term = 0; term < s.terms.n; ++term) {
    const int pa = s.terms.a[term], pb = s.terms.b[term];
    for (int ks = tile.k_begin; ks < tile.k_end; ++ks) {
      if (!tc_wait(&sh.empty[r.stage], r.phase ^ 1, &sh.stop)) return false;
      unsigned char* sa = ring + r.stage * kTcStageBytes;
      unsigned char* sb = sa + kTcABytes;
      const uint32_t bar = in_first(&sh.full[r.stage]);
      // both CTAs' bytes (the other's may land first: the phase ends with
      // this arrival at the earliest)
      if (rank == 0) mbar_arrive_expect_tx(&sh.full[r.stage], 2 * kTcStageBytes);
      const int k0 = ks * kTcK;
      if constexpr (Job::A_MN) {
#pragma unroll
        for (int i = 0; i < kTcRows / 64; ++i) tma_load_3d(sa + i * kTcK * 128, ma, m0 + 64 * i, k0, pa, bar);
      } else {
        tma_load_3d(sa, ma, k0, m0, pa, bar);
      }
      if constexpr (Job::B_MN) {
#pragma unroll
        for (int i = 0; i < kTcN / 2 / 64; ++i)
          tma_load_3d(sb + i * kTcK * 128, mb, n0 + 64 * i, s.b_k0 + k0, pb, bar);
      } else {
        tma_load_3d(sb, mb, s.b_k0 + k0, n0, pb, bar);
      }
      r.next();
    }
  }
  return true;
}

// Matrix instructions of one tile; false once a wait has given up.
template <class Job>
__device__ __forceinline__ bool tc_mma_tile(const Job& job, const TcWalk& walk, int64_t t, uint32_t tmem, TcShared& sh,
                                            unsigned char* ring, TcRing& r, TcAcc& acc) {
  const TcTile tile = walk.at(t, job.s);
  const int stages = tile.k_end - tile.k_begin, steps = stages * job.s.terms.n;
  // (no steps: the epilogue takes zeros and waits for nothing)
  for (int at = 0; at < steps;) {
    const int group_end = tc_group_end<Job::GROUP>(at, stages, job.s.terms.n);
    if (!tc_wait(&sh.acc_empty[acc.buf], acc.phase ^ 1, &sh.stop)) return false;
    tc_fence_after();
    const uint32_t d = tmem + acc.buf * kTcN;
    for (bool fresh = true; at < group_end; ++at) {
      if (!tc_wait(&sh.full[r.stage], r.phase, &sh.stop)) return false;
      tc_fence_after();
      const uint32_t sa = smem_u32(ring + r.stage * kTcStageBytes);
      const uint64_t da = tc_desc<Job::A_MN>(sa), db = tc_desc<Job::B_MN>(sa + kTcABytes);
#pragma unroll
      for (int k = 0; k < kTcK / 16; ++k)
        tc_mma(d, da + k * kTcStepK<Job::A_MN>, db + k * kTcStepK<Job::B_MN>, kTcInstr<Job::A_MN, Job::B_MN>,
               !fresh || k > 0);
      fresh = false;
      tc_commit(&sh.empty[r.stage]);
      r.next();
    }
    tc_commit(&sh.acc_full[acc.buf]);
    acc.next();
  }
  return true;
}

// Epilogue of one tile by the eight epilogue warps; false once a wait has
// given up (one verdict for the warp: the TMEM loads need all its lanes).
template <class Job>
__device__ __forceinline__ bool tc_finish_tile(const Job& job, const TcWalk& walk, int64_t t, int rank, uint32_t tmem,
                                               TcShared& sh, float* block, TcAcc& acc) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp & 3, half = warp >> 2;
  const uint32_t src0 = tmem + ((uint32_t)(quarter * 32) << 16) + half * (kTcN / 2);
  const auto ready = [&] {
    if (!__all_sync(0xffffffffu, tc_wait(&sh.acc_full[acc.buf], acc.phase, &sh.stop))) return false;
    tc_fence_after();
    return true;
  };
  const auto done = [&] {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_cluster(in_first(&sh.acc_empty[acc.buf]));
    acc.next();
  };
  const TcTile tile = walk.at(t, job.s);
  const int stages = tile.k_end - tile.k_begin, steps = stages * job.s.terms.n;
  const int col0 = tile.n0 + half * (kTcN / 2);
  typename Job::Epi::State st;
  job.epi.begin(st, walk, tile, tile.m0 + rank * kTcRows + quarter * 32 + lane, col0);
  if (Job::GROUP == 0 && steps > 0) {
    // straight from TMEM, 32 columns worked on while the next are loaded
    float v[32], w[32];
    if (!ready()) return false;
    const uint32_t src = src0 + acc.buf * kTcN;
    tc_load32(src, v);
#pragma unroll 1
    for (int c = 0; c < kTcN / 2; c += 64) {
      tc_load_wait(v);
      tc_load32(src + c + 32, w);
      job.epi.chunk(st, col0 + c, v, block);
      tc_load_wait(w);
      if (c + 64 < kTcN / 2) tc_load32(src + c + 64, v);
      else done();
      job.epi.chunk(st, col0 + c + 32, w, block);
    }
  } else if (Job::GROUP == 0) {
    float v[32];
#pragma unroll 1
    for (int c = 0; c < kTcN / 2; c += 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
      job.epi.chunk(st, col0 + c, v, block);
    }
  } else {
    float sum[kTcN / 64][32];
#pragma unroll
    for (int c = 0; c < kTcN / 64; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) sum[c][i] = 0.f;
    for (int at = 0; at < steps; at = tc_group_end<Job::GROUP>(at, stages, job.s.terms.n)) {
      if (!ready()) return false;
#pragma unroll
      for (int c = 0; c < kTcN / 64; ++c) {
        tc_add16(src0 + acc.buf * kTcN + 32 * c, sum[c]);
        tc_add16(src0 + acc.buf * kTcN + 32 * c + 16, sum[c] + 16);
      }
      done();
    }
#pragma unroll
    for (int c = 0; c < kTcN / 64; ++c) job.epi.chunk(st, col0 + 32 * c, sum[c], block);
  }
  job.epi.end(st);
  return true;
}

// The tiles of one product, or of two that do not depend on each other (the
// second's after the first's), dealt to the clusters in turn.
template <class Job1, class Job2>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
    tc_product_kernel(const __grid_constant__ Job1 j1, const __grid_constant__ Job2 j2) {
  constexpr bool two = !std::is_same_v<Job2, TcNoJob>;
  constexpr bool shares = kTcShares<Job1, Job2>;
  extern __shared__ unsigned char tc_smem_raw[];
  __shared__ __align__(8) TcShared sh;
  unsigned char* ring = reinterpret_cast<unsigned char*>(((uintptr_t)tc_smem_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();

  pdl_trigger();
  if (warp == kTcEpiWarps + 1) tc_alloc(&sh.tmem_base, 2 * kTcN);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTcStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], 2 * kTcEpiWarps);
    }
    mbar_init(&sh.drained, 1);
    sh.stop = 0;
    mbar_fence_init();
  }
  if (threadIdx.x == 32 * kTcEpiWarps) {
    tma_prefetch_map(&j1.a);
    tma_prefetch_map(&j1.b);
    if constexpr (two) {
      tma_prefetch_map(&j2.a);
      tma_prefetch_map(&j2.b);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  pdl_wait();
  const TcWalk w1(j1.s);
  const auto second = [&] {
    if constexpr (two) return TcWalk(j2.s);
    else return w1;
  };
  const TcWalk w2 = second();
  const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1, end = w1.tiles + (two ? w2.tiles : 0);
  // f(job, walk, tile) for this cluster's tiles until it returns false
  const auto each_tile = [&](auto&& f) {
    for (int64_t t = first; t < end; t += step) {
      if (t < w1.tiles) {
        if (!f(j1, w1, t)) return;
      } else if constexpr (two) {
        if (!f(j2, w2, t - w1.tiles)) return;
      }
    }
  };

  TcRing copied;  // where the copies' thread has stopped
  // (without partial sums the launch's registers are enough)
  if (warp >= kTcEpiWarps + 2) {
    // ---- idle ----
    if constexpr (shares) regs_give<kTcIssueRegs>();
  } else if (warp == kTcEpiWarps) {
    // ---- copies ----
    if constexpr (shares) regs_give<kTcIssueRegs>();
    if (lane == 0) {
      // operands written by earlier kernels' ordinary stores, read by copies
      asm volatile("fence.proxy.async;" ::: "memory");
      each_tile([&](const auto& job, const TcWalk& w, int64_t t) { return tc_copy_tile(job, w, t, rank, sh, ring, copied); });
    }
  } else if (warp == kTcEpiWarps + 1) {
    // ---- matrix instructions ----
    if constexpr (shares) regs_give<kTcIssueRegs>();
    if (lane == 0 && rank == 0) {
      TcRing r;
      TcAcc acc;
      each_tile([&](const auto& job, const TcWalk& w, int64_t t) { return tc_mma_tile(job, w, t, tmem, sh, ring, r, acc); });
      tc_commit(&sh.drained);
    }
  } else {
    // ---- epilogue ----
    if constexpr (shares) regs_take<kTcEpiRegs>();
    TcAcc acc;
    float* block = reinterpret_cast<float*>(ring + kTcStages * kTcStageBytes) + warp * kTcBlockFloats;
    each_tile([&](const auto& job, const TcWalk& w, int64_t t) { return tc_finish_tile(job, w, t, rank, tmem, sh, block, acc); });
  }
  // The roles of both CTAs have ended: nothing more is issued, and what is
  // still in flight is over shortly (a wait that began with the role would
  // have to last as long as the other CTA's, the whole product).
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  // Every copy lands before the cluster ends (when all went well the matrix
  // instructions have waited for it too).  Stage i was last filled in
  // copied.phase if i < copied.stage, else in the phase before, or never:
  // that wait returns at once.
  if (threadIdx.x == 32 * kTcEpiWarps && rank == 0)
    for (int i = 0; i < kTcStages; ++i)
      mbar_wait_bounded(&sh.full[i], i < copied.stage ? copied.phase : copied.phase ^ 1);
  // whatever was issued completes before TMEM is freed (in both CTAs: no
  // arrival is still on its way when the cluster ends)
  if (threadIdx.x == 32 * (kTcEpiWarps + 1)) mbar_wait_bounded(&sh.drained, 0);
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == kTcEpiWarps + 1) tc_free(tmem, 2 * kTcN);
}

}  // namespace rlca
