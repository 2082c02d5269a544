// Matrix product of e4m3 operands with fp32 scales for blocks of 128:
//
//   out[m, n] = sum_b sa[b, m] * sw[n / 128, b] * sum_{k in block b} a[m, k] * w[n, k]
//
// dense (one weight matrix) or grouped by expert (rows offsets[e] ..
// offsets[e+1]-1 use the weights of expert e).
//
// One 128-wide block of k is one 128-byte swizzled row of both operands: TMA fills
// a ring of stages, four kind::f8f6f4 MMAs reduce the block into a TMEM buffer,
// and the epilogue warps read the buffer and add it, times the block's scales, to
// fp32 sums in registers while the next blocks run into the other buffers.
//
// Three forms of tile, chosen by an estimate of the time (at the end):
//   swapped  128 weight rows x 16, 32 or 64 tokens, k split over a cluster where
//            there are few tiles: the weights are the M operand of tcgen05.mma
//            and the tokens its N operand, so that a handful of tokens wastes no
//            tensor-core rows and streams the weights once;
//   square   128 tokens x 128 weight rows, one CTA;
//   paired   256 tokens x 256 weight rows, a pair of CTAs (cta_group::2).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "mla_internal.h"
#include "per_device.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace gemm8 {

using namespace ptx;

__device__ int g_gemm_error;

constexpr int kBlockK = 128;     // k columns per scale block = bytes of one swizzled operand row
constexpr int kTileRows = 128;   // weight rows per tile = columns that share a weight scale
constexpr int kMaxExperts = 1024;
constexpr long long kTimeoutCycles = 2000000000LL;  // about a second: a wait this long has failed

struct Args {
  const float* a_scales;  // [k blocks][a_scale_stride]
  const float* w_scales;  // [experts][row blocks][k blocks]
  const int32_t* offsets; // int32 [experts + 1], nullptr: one group of all rows
  void* out;
  int64_t a_scale_stride, ldo;
  int m, n, k_blocks, row_blocks, experts;  // row_blocks: tiles along the weight rows
  int scale_rows;  // 128-row blocks of the weights' scales
  int splits;  // CTAs that share a tile's k blocks (a cluster); 1: none
  int give_up; // epilogue warp of CTA 0 that gives up at once (tests of the swapped form); -1: none
};

template <int TN, bool kSplit>
struct Cfg {
  // warps: 0 TMA, 1 MMA, then 4 (one per TMEM lane quadrant) or 8 (two, each
  // with half of the tokens) of the epilogue, then the scales
  static constexpr int kEpiWarps = TN >= 32 ? 8 : 4;
  static constexpr int kThreads = 32 * (kEpiWarps + 3);
  static constexpr int kStageA = kTileRows * kBlockK;  // weights
  static constexpr int kStageB = TN * kBlockK;         // tokens
  static constexpr int kStage = kStageA + kStageB;
  // partial sums received from the CTAs of a split tile: [source][row][token slice]
  static constexpr int kRecv = kSplit ? kTileRows * TN * 4 : 0;
  // Two CTAs share an SM: twice the places for clusters (36 of 8 fit instead of
  // 15), and one CTA loads while the other exchanges.
  static constexpr int kCtasPerSm = 2;
  static constexpr int kRing = 106 * 1024 - kRecv;
  static constexpr int kStages = kRing / kStage < 8 ? kRing / kStage : 8;
  static constexpr int kScaleStages = 8;
  static constexpr int kScaleSlot = TN + 4;            // token scales, then the weights' scale
  static constexpr int kBufs = 4;
  static constexpr uint32_t kTmemCols = kBufs * TN;
  static constexpr int kOffRecv = kStages * kStage;
  static constexpr int kOffScales = kOffRecv + kRecv;
  static constexpr int kOffPrefix = kOffScales + kScaleStages * kScaleSlot * 4;
  static constexpr int kOffBars = kOffPrefix + (kMaxExperts + 8) * 4;
  static constexpr int kSmem = kOffBars + 512 + 1024;  // + alignment slack
};

struct Bars {
  uint32_t base;
  __device__ uint32_t full(int s) const { return base + 8 * s; }
  __device__ uint32_t empty(int s) const { return base + 8 * (16 + s); }
  __device__ uint32_t sfull(int s) const { return base + 8 * (32 + s); }
  __device__ uint32_t sempty(int s) const { return base + 8 * (40 + s); }
  __device__ uint32_t tfull(int s) const { return base + 8 * (48 + s); }
  __device__ uint32_t tempty(int s) const { return base + 8 * (52 + s); }
  __device__ uint32_t fin() const { return base + 8 * 56; }
  __device__ uint32_t recv() const { return base + 8 * 57; }
};

// Position in a ring of N slots: the slot, and the parity of its current pass.
// A barrier is waited for at `phase` by the reader of its slot, and at
// `phase ^ 1` by the writer (which passes at once in the first pass).
template <int N>
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ uint32_t flag_load(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void flag_store(uint32_t addr, uint32_t v) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Bounded wait; false: gave up here or elsewhere in the CTA (the flag in shared memory).
template <bool kCluster = false>
__device__ __forceinline__ bool wait_bar(uint32_t abort_flag, uint32_t bar, uint32_t parity, int code) {
  if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (flag_load(abort_flag)) return false;
    if (clock64() - t0 > kTimeoutCycles) {
      flag_store(abort_flag, 1);
      atomicCAS(&g_gemm_error, 0, code);
      return false;
    }
  }
}
template <bool kCluster = false>
__device__ __forceinline__ bool wait_bar_warp(uint32_t abort_flag, uint32_t bar, uint32_t parity, int code) {
  const bool ok = wait_bar<kCluster>(abort_flag, bar, parity, code);
  return __all_sync(0xffffffffu, ok);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// wait_bar_warp for the issuing warps.  The first tries loop inside one
// statement and the verdict is a vote, so the compiler sees no divergence and
// keeps the ring's state, the descriptors and the branch in uniform registers.
__device__ __forceinline__ bool wait_bar_uniform(uint32_t abort_flag, uint32_t bar, uint32_t parity, int code) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
      "TRY:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 64;\n\t@q bra TRY;\n"
      "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, ok)) return true;
  return wait_bar_warp(abort_flag, bar, parity, code);
}

// Wait at a role's end: limited, without a verdict.
__device__ __forceinline__ void wait_limited(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity) && clock64() - t0 < kTimeoutCycles) {
  }
}
// The last `issued` (at most N) uses of the producer's ring are released.
template <int N>
__device__ __forceinline__ void drain(Ring<N> ring, int issued, const Bars& bars) {
  const long long t0 = clock64();
  for (int k = 0; k < N; ++k, ring.next()) {  // from the oldest slot on
    if (k < N - issued) continue;             // never used
    while (!mbar_try_wait(bars.empty(ring.slot), ring.phase ^ 1) && clock64() - t0 < kTimeoutCycles) {
    }
  }
}

// Shared-memory operand descriptors here differ in the start address alone (the
// low word): rows of 128 bytes in the 128-byte swizzle, groups of 8 rows 1 KB
// apart.  The issuing thread adds to the low word instead of building each
// descriptor, which is most of its work per k block.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (kSwizzle128B << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }

// The four K = 32 products of a 128-wide k block: D[tmem] = A[smem] * B[smem]^T,
// 8-bit operands; a, b: low words.  Issued where `go` is nonzero: predicated
// instructions, so that a whole warp runs through without a branch.
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t go) {
  asm volatile(
      "{\n\t.reg .pred g, p;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\t"
      "setp.ne.b32 g, %4, 0;\n\tsetp.ne.b32 p, 0, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "@g tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 da, {x, %5};\n\tmov.b64 db, {y, %5};\n\t"
      "@g tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 da, {x, %5};\n\tmov.b64 db, {y, %5};\n\t"
      "@g tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 da, {x, %5};\n\tmov.b64 db, {y, %5};\n\t"
      "@g tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(go), "r"(kDescHigh)
      : "memory");
}
// Arrive on `bar` when the products issued so far are done (where `go`).
__device__ __forceinline__ void mma_commit_if(uint32_t bar, uint32_t go) {
  asm volatile(
      "{\n\t.reg .pred g;\n\tsetp.ne.b32 g, %1, 0;\n\t"
      "@g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(go)
      : "memory");
}
// fp32 accumulator, e4m3 x e4m3, both K-major
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
// Shared memory of this CTA -> shared memory of a CTA of the cluster, completing
// `bytes` on that CTA's barrier (remote addresses from mapa).
__device__ __forceinline__ void bulk_copy_cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t mbar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(mbar)
               : "memory");
}
// 4-byte asynchronous copy; bytes == 0 writes zeros and reads nothing
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// this thread's earlier cp.async copies arrive on `bar` when they have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// Copies from shared to global memory: a box, the end of a group, the waits until
// at most kPending groups still read and until all are done.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// threadIdx.x, read where it stands: what is computed from it is not moved out of loops
__device__ __forceinline__ int thread_index() {
  int v;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(v));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  union U { float2 f; uint64_t u; } x, y, z, d;
  x.f = a; y.f = b; z.f = c;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.u) : "l"(x.u), "l"(y.u), "l"(z.u));
  return d.f;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  union U { float2 f; uint64_t u; } x, y, d;
  x.f = a; y.f = b;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(x.u), "l"(y.u));
  return d.f;
}
// 32 lanes x 8 or 16 columns with the wait in the same statement
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Programmatic dependent launch: wait for the kernels before this one in the
// stream to be complete; let the next one start its prologue.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Announce `bytes` on `bar` and load a box that completes them, where `go`.
__device__ __forceinline__ void tma_announce_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t bytes, int x,
                                                  int y, uint32_t go) {
  asm volatile(
      "{\n\t.reg .pred g;\n\tsetp.ne.b32 g, %6, 0;\n\t"
      "@g mbarrier.arrive.expect_tx.shared::cta.b64 _, [%2], %5;\n\t"
      "@g cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(bytes), "r"(go)
      : "memory");
}
__device__ __forceinline__ void tma_load_if(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, uint32_t go) {
  asm volatile(
      "{\n\t.reg .pred g;\n\tsetp.ne.b32 g, %5, 0;\n\t"
      "@g cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(go)
      : "memory");
}

// An issuing warp's way through its k blocks: of kTurns warps that take them in
// turn, `id` has blocks id, id + kTurns, ... of `total`, and with them every
// kTurns-th stage and buffer.  What it waits for is nearly always there, so its
// own instructions set the pace: the whole warp runs the loop and a predicate
// lets one lane issue, the next block's barriers are looked at while this one's
// products go out, and one vote judges both (246 cycles per block alone on an
// SM; 404 with two waits and a branch, 690 by one lane under a branch).
template <int kTurns, int kStages, int kBufs>
__device__ __forceinline__ bool issue_in_turn(uint32_t abort_flag, const Bars& bars, uint32_t a0, uint32_t b0,
                                              uint32_t stage, uint32_t tmem, uint32_t cols, uint32_t idesc, int id,
                                              int64_t total, uint32_t go, int code) {
  static_assert(kStages % kTurns == 0 && kBufs % kTurns == 0, "whole shares");
  Ring<kStages / kTurns> ring;
  Ring<kBufs / kTurns> buf;
  bool full = false, empty = false;
  for (int64_t j = id; j < total; j += kTurns) {
    const uint32_t s = ring.slot * kTurns + id, b = buf.slot * kTurns + id;
    if (!__all_sync(0xffffffffu, full & empty)) {
      // the buffer's release comes last: it is waited for last
      if (!wait_bar_uniform(abort_flag, bars.full(s), ring.phase, code) ||
          !wait_bar_uniform(abort_flag, bars.tempty(b), buf.phase ^ 1, code + 1))
        return false;
    }
    tc_fence_after();
    ring.next();
    buf.next();
    full = mbar_test_wait(bars.full(ring.slot * kTurns + id), ring.phase);
    empty = mbar_test_wait(bars.tempty(buf.slot * kTurns + id), buf.phase ^ 1);
    mma_block(tmem + b * cols, a0 + s * (stage >> 4), b0 + s * (stage >> 4), idesc, go);
    mma_commit_if(bars.empty(s), go);
    mma_commit_if(bars.tfull(b), go);
  }
  return true;
}

// Rows [lo, hi) of expert e, as the offsets say.  Plain loads: the kernel before
// this one may still be writing them while this one is resident, and a read-only
// load may only be used on what nobody writes in a kernel's lifetime.
__device__ __forceinline__ int2 expert_rows(const Args& a, int e) {
  if (a.offsets == nullptr) return make_int2(0, a.m);
  return make_int2(a.offsets[e], a.offsets[e + 1]);
}

// prefix[e] = token tiles of the experts before e, by one warp.  An expert whose
// range is not 0 <= lo <= hi <= m, or begins before the end of an earlier one,
// owns no row (recorded): no access leaves the arrays, no row has two owners, and
// there are no more tiles than most_token_tiles on the host.
template <int TN>
__device__ __forceinline__ void scan_experts(const Args& a, int* prefix, int lane) {
  int run = 0, end = 0;  // tiles, and the last row of a range, so far
  for (int e0 = 0; e0 < a.experts; e0 += 32) {
    const int e = e0 + lane;
    int2 r = make_int2(end, end);
    if (e < a.experts) r = expert_rows(a, e);
    const bool range = r.x >= 0 && r.y >= r.x && r.y <= a.m;
    // a range ends where the next begins: if every one is a range, they ascend
    if (__all_sync(0xffffffffu, range && r.x >= end)) {
      end = __shfl_sync(0xffffffffu, r.y, min(31, a.experts - 1 - e0));
    } else {
      int seen = range && r.y > r.x ? r.y : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, seen, o);
        if (lane >= o) seen = max(seen, v);
      }
      int before = __shfl_up_sync(0xffffffffu, seen, 1);
      before = lane == 0 ? end : max(end, before);
      if (!range || (r.y > r.x && r.x < before)) {
        atomicCAS(&g_gemm_error, 0, 0x701);
        r = make_int2(0, 0);
      }
      end = max(end, __shfl_sync(0xffffffffu, seen, 31));
    }
    const int c = (int)(((int64_t)r.y - r.x + TN - 1) / TN);
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (e < a.experts) prefix[e] = run + inc - c;
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) prefix[a.experts] = run;
}

struct Tile {
  int expert, row_block, tok0, tok_end;
};

// Tile `idx`: experts in order; within an expert the token tiles of one block
// of weight rows are neighbours, so concurrent CTAs read the same weights.
template <int TN>
__device__ __forceinline__ Tile find_tile(const Args& a, const int* prefix, int idx) {
  int e = 0;
  if (a.offsets != nullptr) {
    const int p = idx / a.row_blocks;  // an expert owns prefix[e] .. prefix[e+1] token tiles
    int lo = 0, hi = a.experts - 1;
    while (lo < hi) {  // last e with prefix[e] <= p
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= p) lo = mid; else hi = mid - 1;
    }
    e = lo;
  }
  const int first = prefix[e], count = prefix[e + 1] - first;
  const int rem = idx - first * a.row_blocks;
  const int2 rows = expert_rows(a, e);
  Tile t;
  t.expert = e;
  t.row_block = rem / count;
  t.tok0 = rows.x + (rem - t.row_block * count) * TN;
  t.tok_end = rows.y;
  return t;
}

__device__ __forceinline__ void store_out(const Args& a, bool fp32, int m, int n, float v) {
  if (fp32)
    static_cast<float*>(a.out)[m * a.ldo + n] = v;
  else
    static_cast<__nv_bfloat16*>(a.out)[m * a.ldo + n] = __float2bfloat16_rn(v);
}

// kSplit: the CTAs of a cluster share a tile, each summing its part of the k
// blocks; the sums are then exchanged through distributed shared memory, each
// CTA adding up and storing a slice of the tile's tokens in CTA order (the
// grid holds one cluster per tile).
template <int TN, bool kSplit, bool kFp32>
__global__ void __launch_bounds__(Cfg<TN, kSplit>::kThreads, Cfg<TN, kSplit>::kCtasPerSm)
    gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a, const Args a) {
  using C = Cfg<TN, kSplit>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const Bars bars{sbase + C::kOffBars};
  int* prefix = reinterpret_cast<int*>(smem + C::kOffPrefix);
  const uint32_t abort_flag = sbase + C::kOffPrefix + (kMaxExperts + 4) * 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(prefix + kMaxExperts + 5);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    flag_store(abort_flag, 0);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(bars.full(i), 1);
      mbar_init(bars.empty(i), 1);
    }
    for (int i = 0; i < C::kScaleStages; ++i) {
      mbar_init(bars.sfull(i), 32);
      mbar_init(bars.sempty(i), C::kEpiWarps);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(bars.tfull(i), 1);
      mbar_init(bars.tempty(i), C::kEpiWarps);
    }
    mbar_init(bars.fin(), 1);
    mbar_init(bars.recv(), 1);
    fence_mbar_init();
    if (kSplit) mbar_arrive_expect_tx(bars.recv(), C::kRecv);
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_a);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  const int splits = kSplit ? a.splits : 1;
  const int rank = kSplit ? (int)cluster_ctarank() : 0;
  const int first = kSplit ? (int)blockIdx.x / splits : (int)blockIdx.x;
  const int kb0 = kSplit ? (int)((int64_t)a.k_blocks * rank / splits) : 0;
  const int kb1 = kSplit ? (int)((int64_t)a.k_blocks * (rank + 1) / splits) : a.k_blocks;
  if (warp == 0 && lane == 0 && a.offsets == nullptr) {
    // pull the first weights into L2 while the kernel before this one drains
    // (a hint: the loads that follow the wait below read what is there then)
    const int wrow = first / ((a.m + TN - 1) / TN) * kTileRows;
    for (int kb = kb0; kb < min(kb0 + C::kStages, kb1); ++kb) tma_prefetch_2d(&tm_w, kb * kBlockK, wrow);
  }
  // all of the above overlaps the kernel before; nothing of its results, or of
  // what it still reads, is touched before this returns
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 2) scan_experts<TN>(a, prefix, lane);
  // every warp whole again before each .aligned instruction (the barriers, the
  // TMEM calls): executed by parts of a warp they are undefined
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (kSplit) cluster_sync();  // the peers' barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const int tiles = prefix[a.experts] * a.row_blocks;
  const int step = kSplit ? tiles : (int)gridDim.x;  // a split grid has a cluster for every tile

  if (warp == 0) {
    // ---- TMA producer
    if (lane == 0) {
      int j = 0;
      Ring<C::kStages> ring;
      bool ok = true;
      for (int idx = first; ok && idx < tiles; idx += step) {
        const Tile t = find_tile<TN>(a, prefix, idx);
        const int wrow = t.expert * a.n + t.row_block * kTileRows;
        for (int kb = kb0; kb < kb1; ++kb, ++j, ring.next()) {
          const uint32_t s = ring.slot;
          if (!wait_bar(abort_flag, bars.empty(s), ring.phase ^ 1, 0x711)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bars.full(s), C::kStage);
          tma_load_2d(sbase + s * C::kStage, &tm_w, bars.full(s), kb * kBlockK, wrow);
          tma_load_2d(sbase + s * C::kStage + C::kStageA, &tm_a, bars.full(s), kb * kBlockK, t.tok0);
        }
      }
      // the copies in flight, and the arrivals that release their stages, must
      // have landed before the CTA leaves
      drain<C::kStages>(ring, j, bars);
    }
  } else if (warp == 1) {
    // ---- MMA issuer
    const uint32_t go = elect_one();
    const int64_t mine = tiles > first ? (tiles - first + step - 1) / step : 0;
    issue_in_turn<1, C::kStages, C::kBufs>(abort_flag, bars, desc_low(sbase), desc_low(sbase + C::kStageA), C::kStage, tmem,
                                           TN, idesc_e4m3(kTileRows, TN), 0, mine * (kb1 - kb0), go, 0x712);
    mma_commit_if(bars.fin(), go);  // everything issued is done before TMEM is released
    if (go) wait_limited(bars.fin(), 0);
  } else if (warp == C::kEpiWarps + 2) {
    // ---- scales of each k block into their own ring: a load per block on the
    // epilogue's path would cost it a memory latency per block
    Ring<C::kScaleStages> ring;
    bool ok = true;
    for (int idx = first; ok && idx < tiles; idx += step) {
      const Tile t = find_tile<TN>(a, prefix, idx);
      const float* sw = a.w_scales + ((int64_t)t.expert * a.scale_rows + t.row_block) * a.k_blocks;
      for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
        const uint32_t s = ring.slot;
        if (!wait_bar_warp(abort_flag, bars.sempty(s), ring.phase ^ 1, 0x714)) {
          ok = false;
          break;
        }
        const float* src = a.a_scales + kb * a.a_scale_stride + t.tok0;
        const uint32_t dst = sbase + C::kOffScales + s * C::kScaleSlot * 4;
        for (int i = lane; i < TN; i += 32) {
          const bool in = t.tok0 + i < t.tok_end;
          cp_async4(dst + i * 4, in ? src + i : a.a_scales, in ? 4 : 0);
        }
        if (lane == 0) cp_async4(dst + TN * 4, sw + kb, 4);
        cp_async_arrive(bars.sfull(s));
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---- epilogue: thread = weight row, registers = tokens
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    constexpr int kCols = TN / (C::kEpiWarps / 4);  // tokens of this warp
    const int half = (warp - 2) >> 2;
    const int col0 = half * kCols;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    Ring<C::kScaleStages> ring;
    Ring<C::kBufs> buf;
    bool ok = true;
    if (blockIdx.x == 0 && warp - 2 == a.give_up) {
      flag_store(abort_flag, 1);
      atomicCAS(&g_gemm_error, 0, 0x718);
      ok = false;
    }
    // a warp that has given up still goes through a split tile (there is one)
    for (int idx = first; (ok || kSplit) && idx < tiles; idx += step) {
      const Tile t = find_tile<TN>(a, prefix, idx);
      float2 acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb = kb0; ok && kb < kb1; ++kb, ring.next(), buf.next()) {
        const uint32_t s = ring.slot, b = buf.slot;
        if (!wait_bar_warp(abort_flag, bars.sfull(s), ring.phase, 0x715) ||
            !wait_bar_warp(abort_flag, bars.tfull(b), buf.phase, 0x716)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float* slot = reinterpret_cast<const float*>(smem + C::kOffScales) + s * C::kScaleSlot;
        const float4* sc = reinterpret_cast<const float4*>(slot + col0);
        const float2 w2 = make_float2(slot[TN], slot[TN]);
        auto add4 = [&](int c, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
          const float4 s4 = sc[c / 4];
          const float2 s01 = mul2(make_float2(s4.x, s4.y), w2), s23 = mul2(make_float2(s4.z, s4.w), w2);
          acc[c / 2] = fma2(make_float2(__uint_as_float(r0), __uint_as_float(r1)), s01, acc[c / 2]);
          acc[c / 2 + 1] = fma2(make_float2(__uint_as_float(r2), __uint_as_float(r3)), s23, acc[c / 2 + 1]);
        };
        constexpr int kChunk = kSplit && kCols == 32 ? 8 : 16;  // few at a time: two CTAs share the register file
#pragma unroll
        for (int c = 0; c < kCols; c += kChunk) {
          uint32_t r[kChunk];
          tmem_ld(taddr + b * TN + c, r);
#pragma unroll
          for (int i = 0; i < kChunk; i += 4) add4(c + i, r[i], r[i + 1], r[i + 2], r[i + 3]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bars.tempty(b));
          mbar_arrive(bars.sempty(s));
        }
      }
      if (!kSplit && !ok) break;
      const int n = t.row_block * kTileRows + row;
      if (kSplit) {
        // tokens [p * slice, (p + 1) * slice) go to CTA p of the cluster: staged
        // as [token][row] in the ring (idle: the tile's last product has been
        // read) and moved by the copy engine, one contiguous piece per CTA
        const int slice = TN / splits;
        if (ok) {
          float* stage = reinterpret_cast<float*>(smem) + col0 * kTileRows + row;
#pragma unroll
          for (int i = 0; i < kCols; ++i) stage[i * kTileRows] = (i & 1) ? acc[i / 2].y : acc[i / 2].x;
          fence_proxy_async_smem();
        }
        __syncwarp();
        // The barrier has no time limit: every epilogue warp comes here once,
        // whether its waits succeeded or not, and every CTA sends its pieces, so
        // that no peer waits for one in vain (what they hold after a wait that
        // timed out is of no use, which the error word says).
        named_bar_sync(1, 32 * C::kEpiWarps);
        if (warp == 2 && lane < splits) {
          const uint32_t bytes = (uint32_t)slice * kTileRows * 4;
          bulk_copy_cluster(mapa(sbase + C::kOffRecv + rank * bytes, lane), sbase + lane * bytes, bytes,
                            mapa(bars.recv(), lane));
        }
        if (!ok || !wait_bar_warp<true>(abort_flag, bars.recv(), 0, 0x717)) {
          wait_limited(bars.recv(), 0);  // the peers' pieces land before the CTA leaves
          ok = false;
          break;
        }
        const float* recv = reinterpret_cast<const float*>(smem + C::kOffRecv) + row;
        for (int i0 = half * 2; i0 < slice; i0 += 2 * C::kEpiWarps / 4) {  // slices are even
          float v0 = 0.f, v1 = 0.f;
#pragma unroll 4
          for (int p = 0; p < splits; ++p) {
            v0 += recv[(p * slice + i0) * kTileRows];
            v1 += recv[(p * slice + i0 + 1) * kTileRows];
          }
          const int m = t.tok0 + rank * slice + i0;
          if (n < a.n && m < t.tok_end) store_out(a, kFp32, m, n, v0);
          if (n < a.n && m + 1 < t.tok_end) store_out(a, kFp32, m + 1, n, v1);
        }
      } else if (n < a.n) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const int m = t.tok0 + col0 + i;
          if (m < t.tok_end) store_out(a, kFp32, m, n, (i & 1) ? acc[i / 2].y : acc[i / 2].x);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
  if (kSplit) {
    // no peer may still address this CTA's shared memory; nothing is published
    // here, so the arrival need not wait for the output's stores
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  }
}

// The warp's 32 rows x 64 columns of results, kBytes of each row at a time through
// shared memory (in the order of a TMA swizzle) and from there by TMA, which
// drains while the next tile is computed.  kPart: which of a tile's calls; the
// pieces go through the warp's buffers in turn.  Stored by the warps themselves
// the results cost a paired tile 1.9 us, since every SM stores at once: 8192 tokens,
// n 8192, k 2048 134 us, 122 with one buffer and five stages, 119 with two and four.
// A piece that TMA cannot cut (its last rows are the next expert's, or rows that are
// no multiple of 16 bytes) is read back along the rows, by the widest words that the
// rows' alignment allows: 4096 x 4095 x 1024 31 us (4096 x 4096 23 us; 16 bytes of a row
// per lane, stored one by one: 80 us).
template <int kBytes, int kBuffers, int kPart, bool kFp32, bool kVec>
__device__ __forceinline__ void store_tile(const Args& a, const CUtensorMap* tm_out, uint32_t buffers, int m0, int tok_end,
                                           int n0, int lane, const float2 (&acc)[32]) {
  constexpr int kElt = kFp32 ? 4 : 2, kPiece = kBytes / kElt, kPer16 = 16 / kElt, kChunks = kBytes / 16;
  auto swizzled = [](int row, int c) { return row * kBytes + ((c ^ (kBytes == 128 ? row & 7 : (row >> 1) & 3)) << 4); };
#pragma unroll
  for (int p = 0; p < 64 / kPiece; ++p) {
    const uint32_t staging = buffers + (kPart * (64 / kPiece) + p) % kBuffers * (32 * kBytes);
    if (kVec && lane == 0) bulk_wait_read<kBuffers - 1>();
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint32_t at = staging + swizzled(lane, c);
      if (kFp32) {  // pairs, as the sums are held
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 x = acc[(p * kPiece + 4 * c) / 2 + i];
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at + 8 * i), "f"(x.x), "f"(x.y) : "memory");
        }
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = acc[(p * kPiece + 8 * c) / 2 + i];
          __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
          w[i] = *reinterpret_cast<uint32_t*>(&b);
        }
        st_shared_v4(at, make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
    const int n = n0 + p * kPiece;
    // whole boxes, or cut at the array's end; along a row TMA cuts at 16 bytes
    const bool rows = m0 + 32 <= tok_end || tok_end == a.m, cols = n + kPiece <= a.n || a.n % kPer16 == 0;
    if (kVec && rows && cols) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && m0 < tok_end && n < a.n) tma_store_2d(tm_out, staging, n * kElt, m0);
    } else {
      __syncwarp();
      const int last = min(32, tok_end - m0), left = a.n - n;
      uint8_t* dst = static_cast<uint8_t*>(a.out) + (m0 * a.ldo + n) * kElt;
      const int64_t pitch = a.ldo * kElt;
      if (kVec && cols) {
        const int chunk = lane % kChunks;
#pragma unroll 2
        for (int row = lane / kChunks; row < last; row += 32 / kChunks)
          if (chunk * kPer16 < left)
            *reinterpret_cast<uint4*>(dst + row * pitch + chunk * 16) = ld_shared_v4(staging + swizzled(row, chunk));
      } else if (kFp32 || (a.ldo % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % 4 == 0)) {
        // neighbouring lanes store neighbouring 4 bytes: a value, or two
        constexpr int kWords = kBytes / 4, kRows = 32 / kWords > 0 ? 32 / kWords : 1;
#pragma unroll
        for (int word = lane % kWords; word < kWords; word += 32)
#pragma unroll 4
          for (int row = lane / kWords; row < last; row += kRows) {
            const uint32_t v = ld_shared_u32(staging + swizzled(row, word / 4) + word % 4 * 4);
            uint8_t* at = dst + row * pitch + word * 4;
            if ((word + 1) * (4 / kElt) <= left)
              *reinterpret_cast<uint32_t*>(at) = v;
            else if (!kFp32 && word * 2 < left)
              *reinterpret_cast<uint16_t*>(at) = (uint16_t)v;
          }
      } else {
#pragma unroll
        for (int c = lane; c < kPiece; c += 32)
          if (c < left)
#pragma unroll 4
            for (int row = 0; row < last; ++row)
              *reinterpret_cast<uint16_t*>(dst + row * pitch + c * 2) =
                  ld_shared_u16(staging + swizzled(row, c / 8) + c % 8 * 2);
      }
    }
    if (kVec && lane == 0) bulk_commit();  // also of nothing: the wait counts pieces
  }
}

// ------------------------------------------------------------------ square tiles

// 128 tokens x 128 weight rows per CTA.  Here the tokens are the M operand, so an
// epilogue thread owns one token and its factor for a k block is one register,
// not one per column.  It reads its 64 columns of a block in two halves, the
// second while the first is added and the next block's first while the second
// is; a buffer is given back as soon as it is read, and four of them keep the
// products ahead.  Two warps issue the products in turn: the instructions of one
// block take an issuing warp about 550 cycles here, the products 256.
// 256 x 8192 x 8192: 22.3 us (swapped tiles of 64 tokens 42 us, paired 35 us; the
// weights alone 10.6 us); 256 x 4096 x 4096: 13.0 us (16.4, 20.1).
namespace square {

constexpr int kTileTok = 128, kTileCol = 128;
constexpr int kStageTok = kTileTok * kBlockK;
constexpr int kStage = kStageTok + kTileCol * kBlockK;
constexpr int kStages = 6;
constexpr int kScaleGroup = 4;                 // k blocks whose scales share a slot (and a wait)
constexpr int kScaleStages = 4;
constexpr int kScaleRow = kTileTok + 4;        // token scales, then the weights' scale
constexpr int kScaleSlot = kScaleGroup * kScaleRow;
constexpr int kBufs = 4;                       // of 128 TMEM columns
// warps 0-3: copies, MMA, scales, MMA; 4-11: epilogue, two per TMEM lane quadrant
// with 64 columns each
constexpr int kEpiWarps = 8;
constexpr int kCols = kTileCol / (kEpiWarps / 4);
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kStaging = 32 * 64;              // per epilogue warp: 64 bytes of each of its 32 output rows, swizzled
constexpr int kOffStaging = kStages * kStage;
constexpr int kOffScales = kOffStaging + kEpiWarps * kStaging;
constexpr int kOffPrefix = kOffScales + kScaleStages * kScaleSlot * 4;
constexpr int kOffBars = kOffPrefix + (kMaxExperts + 8) * 4;
constexpr int kSmem = kOffBars + 512 + 1024;

__device__ __forceinline__ Tile find(const Args& a, const int* prefix, int idx) {
  return find_tile<kTileTok>(a, prefix, idx);
}

template <bool kFp32, bool kVec>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_square_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                       const __grid_constant__ CUtensorMap tm_out, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const Bars bars{sbase + kOffBars};
  int* prefix = reinterpret_cast<int*>(smem + kOffPrefix);
  const uint32_t abort_flag = sbase + kOffPrefix + (kMaxExperts + 4) * 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(prefix + kMaxExperts + 5);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    flag_store(abort_flag, 0);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bars.full(i), 1);
      mbar_init(bars.empty(i), 1);
    }
    for (int i = 0; i < kScaleStages; ++i) {
      mbar_init(bars.sfull(i), 32);
      mbar_init(bars.sempty(i), kEpiWarps);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(bars.tfull(i), 1);
      mbar_init(bars.tempty(i), kEpiWarps);
    }
    mbar_init(bars.fin(), 1);
    mbar_init(bars.fin() + 8, 1);
    fence_mbar_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_a);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kBufs * kTileCol);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 2) scan_experts<kTileTok>(a, prefix, lane);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const int tiles = prefix[a.experts] * a.row_blocks;
  const int first = (int)blockIdx.x, step = (int)gridDim.x;

  if (warp < 4) {
    if (warp == 0) {
      // ---- TMA producer
      const uint32_t go = elect_one();
      int j = 0;
      Ring<kStages> ring;
      bool ok = true, free = false;  // the next stage, looked at ahead
      for (int idx = first; ok && idx < tiles; idx += step) {
        const Tile t = find(a, prefix, idx);
        const int wrow = t.expert * a.n + t.row_block * kTileCol;
        for (int kb = 0; kb < a.k_blocks; ++kb, ++j) {
          if (!__all_sync(0xffffffffu, free) &&
              !wait_bar_uniform(abort_flag, bars.empty(ring.slot), ring.phase ^ 1, 0x721)) {
            ok = false;
            break;
          }
          const uint32_t full = bars.full(ring.slot), dst = sbase + ring.slot * kStage;
          ring.next();
          free = mbar_test_wait(bars.empty(ring.slot), ring.phase ^ 1);
          tma_announce_load(dst, &tm_a, full, kStage, kb * kBlockK, t.tok0, go);
          tma_load_if(dst + kStageTok, &tm_w, full, kb * kBlockK, wrow, go);
        }
      }
      if (go) drain<kStages>(ring, j, bars);
    } else if (warp == 1 || warp == 3) {
      // ---- MMA issuers
      const uint32_t go = elect_one();
      const int id = warp >> 1;
      const int64_t mine = tiles > first ? (tiles - first + step - 1) / step : 0;
      issue_in_turn<2, kStages, kBufs>(abort_flag, bars, desc_low(sbase), desc_low(sbase + kStageTok), kStage, tmem,
                                       kTileCol, idesc_e4m3(kTileTok, kTileCol), id, mine * a.k_blocks, go, 0x722);
      mma_commit_if(bars.fin() + 8 * id, go);
      if (go) wait_limited(bars.fin() + 8 * id, 0);
    } else {
      // ---- scales: the tile's tokens and its block of weights
      Ring<kScaleStages> ring;
      bool ok = true;
      for (int idx = first; ok && idx < tiles; idx += step) {
        const Tile t = find(a, prefix, idx);
        const float* sw = a.w_scales + ((int64_t)t.expert * a.scale_rows + t.row_block) * a.k_blocks;
        for (int kb = 0; kb < a.k_blocks; kb += kScaleGroup, ring.next()) {
          if (!wait_bar_warp(abort_flag, bars.sempty(ring.slot), ring.phase ^ 1, 0x724)) {
            ok = false;
            break;
          }
          for (int g = kb; g < min(kb + kScaleGroup, a.k_blocks); ++g) {
            const float* src = a.a_scales + g * a.a_scale_stride + t.tok0;
            const uint32_t dst = sbase + kOffScales + (ring.slot * kScaleSlot + (g - kb) * kScaleRow) * 4;
#pragma unroll
            for (int i = 0; i < kTileTok; i += 32) {
              const bool in = t.tok0 + i + lane < t.tok_end;
              cp_async4(dst + (i + lane) * 4, in ? src + i + lane : a.a_scales, in ? 4 : 0);
            }
            if (lane == 0) cp_async4(dst + kTileTok * 4, sw + g, 4);
          }
          cp_async_arrive(bars.sfull(ring.slot));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---- epilogue: thread = token, registers = 64 weight rows
    const int quad = warp & 3, part = (warp - 4) >> 2;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + part * kCols;
    const uint32_t staging = sbase + kOffStaging + (warp - 4) * kStaging;
    const float* slots = reinterpret_cast<const float*>(smem + kOffScales);
    Ring<kScaleStages> ring;
    Ring<kBufs> buf;
    bool ok = true;
    for (int idx = first; ok && idx < tiles; idx += step) {
      const Tile t = find(a, prefix, idx);
      const int m0 = t.tok0 + quad * 32;
      float2 acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      ok = wait_bar_warp(abort_flag, bars.sfull(ring.slot), ring.phase, 0x725) &&
           wait_bar_warp(abort_flag, bars.tfull(buf.slot), buf.phase, 0x726);
      if (!ok) break;
      const float* slot = slots + ring.slot * kScaleSlot;
      float f = slot[quad * 32 + lane] * slot[kTileTok];
      uint32_t r0[32], r1[32];
      tc_fence_after();
      tmem_ld32_async(taddr + buf.slot * kTileCol, r0);
      for (int kb = 0; kb < a.k_blocks; ++kb) {
        float2 f2 = make_float2(f, f);
        tmem_wait_ld32(r0);
        tmem_ld32_async(taddr + buf.slot * kTileCol + 32, r1);
        // the next block: its product, looked at, and its factor
        const bool more = kb + 1 < a.k_blocks;
        const uint32_t release = bars.tempty(buf.slot);
        buf.next();
        const bool there = mbar_test_wait(bars.tfull(buf.slot), buf.phase);
        if ((kb & (kScaleGroup - 1)) == kScaleGroup - 1 || !more) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.sempty(ring.slot));
          ring.next();
          if (more && !wait_bar_warp(abort_flag, bars.sfull(ring.slot), ring.phase, 0x725)) ok = false;
          slot = slots + ring.slot * kScaleSlot;
        } else {
          slot += kScaleRow;
        }
        f = slot[quad * 32 + lane] * slot[kTileTok];  // (past the last block: not used)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          acc[i] = fma2(make_float2(__uint_as_float(r0[2 * i]), __uint_as_float(r0[2 * i + 1])), f2, acc[i]);
        tmem_wait_ld32(r1);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(release);
        if (!ok) break;
        if (more) {
          if (!__all_sync(0xffffffffu, there) && !wait_bar_warp(abort_flag, bars.tfull(buf.slot), buf.phase, 0x726)) {
            ok = false;
            break;
          }
          tc_fence_after();
          tmem_ld32_async(taddr + buf.slot * kTileCol, r0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          acc[16 + i] = fma2(make_float2(__uint_as_float(r1[2 * i]), __uint_as_float(r1[2 * i + 1])), f2, acc[16 + i]);
      }
      if (!ok) break;
      store_tile<64, 1, 0, kFp32, kVec>(a, &tm_out, staging, m0, t.tok_end, t.row_block * kTileCol + part * kCols, lane,
                                        acc);
    }
    if (kVec && lane == 0) bulk_wait();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kBufs * kTileCol);
}

}  // namespace square

// ------------------------------------------------------------------ paired tiles

// A pair of CTAs (cta_group::2) computes 256 tokens x 256 weight rows: the tokens
// are the M operand, 128 of them per CTA, so an epilogue thread owns one token.
// Each CTA loads its own 128 tokens and 128 of the weight rows; the pair's tensor
// cores read both, which halves the shared-memory and L2 traffic of a 128 x 256
// tile.
// Additions (256 cycles a block on the FMA pipes) and TMEM reads have to overlap to
// keep up with the products (512).  So the products of a block come in two halves,
// of 64 of each CTA's weight rows, issued by a warp each into buffers of their own,
// and half of the epilogue's warps take each half: they run out of step, and
// within a warp 32 columns are read while 32 are added.  8192 tokens, n = k = 8192:
// 429 us in a burst at 2070 MHz, 2.6 PFLOP/s; 476 in a steady loop, whose power limit
// leaves 1720 MHz (both halves in one product, all warps in step, reads and additions
// in turn: 3 % more; in square tiles 496 where these take 435).  Spills in the
// epilogue's loop cost 4 to 20 %, so it has 216 registers and its state is counted, not
// kept (8 bytes are left with bf16 results, 4 with unaligned fp32 ones, none with fp32
// ones that the copy engine stores).
namespace paired {

constexpr int kTileTok = 256, kTileCol = 256;  // of the pair
constexpr int kHalf = 128;
constexpr int kStage = 2 * kHalf * kBlockK;    // per CTA: tokens, then weights
constexpr int kStages = 4;
constexpr int kScaleGroup = 4;                 // k blocks whose scales share a slot (and a wait)
constexpr int kScaleStages = 4;
constexpr int kScaleRow = kHalf + 4;           // token scales, then two weight scales
constexpr int kScaleSlot = kScaleGroup * kScaleRow;
constexpr int kBufs = 4;                       // of 128 TMEM columns: two for each half
// warps 0-3: TMA, MMA of the first half, scales, MMA of the second; 4-11: epilogue,
// one per TMEM lane quadrant and half
constexpr int kEpiWarps = 8;
constexpr int kCols = kTileCol / (kEpiWarps / 4);
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kRegsLoad = 72, kRegsEpi = 216;  // 128 x 72 + 256 x 216 = 384 x 168, the launch's registers
constexpr int kStaging = 2 * 32 * 128;         // per epilogue warp: twice 128 bytes of each of its 32 output rows, swizzled
constexpr int kOffStaging = kStages * kStage;
constexpr int kOffScales = kOffStaging + kEpiWarps * kStaging;
constexpr int kOffPrefix = kOffScales + kScaleStages * kScaleSlot * 4;
constexpr int kOffBars = kOffPrefix + (kMaxExperts + 8) * 4;
constexpr int kSmem = kOffBars + 512 + 1024;

__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Load into this CTA's shared memory, completing on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs when the products issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// Arrive on a barrier of either CTA of the pair (address from mapa).  Only a
// TMEM buffer's reads precede it, which the tcgen05 fence orders; a release at
// cluster scope would wait for every store in flight (measured: 1000 cycles).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// The tokens of `t` that this CTA holds start at tok0 + 128 * rank.
__device__ __forceinline__ Tile find(const Args& a, const int* prefix, int idx) {
  return find_tile<kTileTok>(a, prefix, idx);  // a.row_blocks counts 256-row tiles here
}

// a.row_blocks: 256-row tiles of the weights; a.scale_rows: 128-row blocks.
// 32 columns of a block's products, times the block's scales, into the sums from kAt on
template <int kAt>
__device__ __forceinline__ void add32(float2 (&acc)[32], const uint32_t (&r)[32], float f) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    acc[kAt + i] =
        fma2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), make_float2(f, f), acc[kAt + i]);
}

template <bool kFp32, bool kVec>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_paired_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                       const __grid_constant__ CUtensorMap tm_out, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const Bars bars{sbase + kOffBars};
  int* prefix = reinterpret_cast<int*>(smem + kOffPrefix);
  const uint32_t abort_flag = sbase + kOffPrefix + (kMaxExperts + 4) * 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(prefix + kMaxExperts + 5);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();

  if (threadIdx.x == 0) {
    flag_store(abort_flag, 0);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bars.full(i), 1);
      mbar_init(bars.empty(i), 2);  // both halves of the products
    }
    for (int i = 0; i < kScaleStages; ++i) {
      mbar_init(bars.sfull(i), 32);
      mbar_init(bars.sempty(i), kEpiWarps);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(bars.tfull(i), 1);
      mbar_init(bars.tempty(i), kEpiWarps);  // both CTAs' epilogues (the leader's barrier)
    }
    mbar_init(bars.fin(), 1);
    mbar_init(bars.fin() + 8, 1);
    fence_mbar_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_a);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc2(smem_u32(tmem_slot), kBufs * kHalf);
    tmem_relinquish2();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 2) scan_experts<kTileTok>(a, prefix, lane);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const int tiles = prefix[a.experts] * a.row_blocks;
  const int first = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
    if (warp == 0 && lane == 0) {
      // ---- TMA producer: both CTAs' copies complete on the leader's barrier
      int j = 0;
      Ring<kStages> ring;
      const uint32_t full0 = mapa(bars.full(0), 0);
      bool ok = true;
      for (int idx = first; ok && idx < tiles; idx += step) {
        const Tile t = find(a, prefix, idx);
        const int wrow = t.expert * a.n + t.row_block * kTileCol + rank * kHalf;
        const int trow = t.tok0 + rank * kHalf;
        for (int kb = 0; kb < a.k_blocks; ++kb, ++j, ring.next()) {
          const uint32_t s = ring.slot;
          if (!wait_bar(abort_flag, bars.empty(s), ring.phase ^ 1, 0x731)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(bars.full(s), 2 * kStage);
          const uint32_t full = full0 + 8 * s;
          tma_load_2d_pair(sbase + s * kStage, &tm_a, full, kb * kBlockK, trow);
          tma_load_2d_pair(sbase + s * kStage + kHalf * kBlockK, &tm_w, full, kb * kBlockK, wrow);
        }
      }
      // The pair's products release the stages by arrivals in both CTAs: a CTA
      // that left before the last ones came in would have them land in the
      // shared memory of whoever runs there next.  (They also follow the copies.)
      drain<kStages>(ring, j, bars);
    } else if ((warp == 1 || warp == 3) && rank == 1) {
      if (lane == 0) wait_limited(bars.fin() + 8 * (warp >> 1), 0);  // the leader's last arrival here
    } else if (warp == 1 || warp == 3) {
      // ---- MMA issuers (the leader's, for the pair), one for each half: the
      // whole warp runs the loop, one lane issues
      const uint32_t half = warp >> 1;
      constexpr uint32_t kIdesc = idesc_e4m3(kTileTok, kHalf);
      const uint32_t ta0 = desc_low(sbase), wa0 = desc_low(sbase + kHalf * kBlockK + half * (kHalf / 2) * kBlockK);
      const bool issuer = elect_one();
      Ring<kStages> ring;
      Ring<2> buf;
      bool ok = true;
      for (int idx = first; ok && idx < tiles; idx += step) {
        for (int kb = 0; ok && kb < a.k_blocks; ++kb, ring.next(), buf.next()) {
          if (!wait_bar_uniform(abort_flag, bars.full(ring.slot), ring.phase, 0x732)) {
            ok = false;
            break;
          }
          const uint32_t b = 2 * buf.slot + half;
          if (!wait_bar_uniform(abort_flag, bars.tempty(b), buf.phase ^ 1, 0x733)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ta = ta0 + ring.slot * (kStage >> 4), wa = wa0 + ring.slot * (kStage >> 4);
          if (issuer) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_f8_pair(tmem + b * kHalf, ta + 2 * kk, wa + 2 * kk, kIdesc, kk > 0);
            mma_commit_pair(bars.empty(ring.slot));
            mma_commit_pair(bars.tfull(b));
          }
          __syncwarp();
        }
      }
      if (issuer) {
        mma_commit_pair(bars.fin() + 8 * half);
        wait_limited(bars.fin() + 8 * half, 0);
      }
    } else if (warp == 2) {
      // ---- scales: this CTA's tokens and the tile's two weight blocks
      Ring<kScaleStages> ring;
      bool ok = true;
      for (int idx = first; ok && idx < tiles; idx += step) {
        const Tile t = find(a, prefix, idx);
        const int trow = t.tok0 + rank * kHalf;
        const int wb = min(2 * t.row_block + (lane & 1), a.scale_rows - 1);
        const float* sw = a.w_scales + ((int64_t)t.expert * a.scale_rows + wb) * a.k_blocks;
        for (int kb = 0; kb < a.k_blocks; kb += kScaleGroup, ring.next()) {
          if (!wait_bar_warp(abort_flag, bars.sempty(ring.slot), ring.phase ^ 1, 0x734)) {
            ok = false;
            break;
          }
          for (int g = kb; g < min(kb + kScaleGroup, a.k_blocks); ++g) {
            const float* src = a.a_scales + g * a.a_scale_stride + trow;
            const uint32_t dst = sbase + kOffScales + (ring.slot * kScaleSlot + (g - kb) * kScaleRow) * 4;
#pragma unroll
            for (int i = 0; i < kHalf; i += 32) {
              const bool in = trow + i + lane < t.tok_end;
              cp_async4(dst + (i + lane) * 4, in ? src + i + lane : a.a_scales, in ? 4 : 0);
            }
            if (lane < 2) cp_async4(dst + (kHalf + lane) * 4, sw + g, 4);
          }
          cp_async_arrive(bars.sfull(ring.slot));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---- epilogue: thread = token, registers = 128 weight rows: 64 of the
    // leader's and 64 of its peer's, which have a weight scale each
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    const int quad = warp & 3, part = (warp - 4) >> 2;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + part * kHalf;
    const uint32_t tempty = mapa(bars.tempty(part), 0);  // the leader's; this half's next buffer at + 16
    const uint32_t slots = sbase + kOffScales;
    uint32_t n = 0, group = 0;  // blocks and groups of scales so far
    bool ok = true;
    for (int idx = first; ok && idx < tiles; idx += step) {
      float2 acc0[kCols / 4], acc1[kCols / 4];
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) acc0[i] = acc1[i] = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int kb = 0; kb < a.k_blocks; ++kb, ++n) {
        const uint32_t ring = group % kScaleStages, buf = n % 2;
        if (kb % kScaleGroup == 0 && !wait_bar_warp(abort_flag, bars.sfull(ring), (group / kScaleStages) & 1, 0x735)) {
          ok = false;
          break;
        }
        const uint32_t slot = slots + (ring * kScaleSlot + (kb % kScaleGroup) * kScaleRow) * 4;
        const float f = ld_shared_f32(slot + (threadIdx.x & 127) * 4);  // this thread's token
        const float f0 = f * ld_shared_f32(slot + kHalf * 4), f1 = f * ld_shared_f32(slot + kHalf * 4 + 4);
        if (!wait_bar_warp(abort_flag, bars.tfull(2 * buf + part), (n / 2) & 1, 0x736)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t src = taddr + buf * (2 * kHalf);
        uint32_t r0[32], r1[32];
        tmem_ld32_async(src, r0);
        tmem_wait_ld32(r0);
        tmem_ld32_async(src + 32, r1);
        add32<0>(acc0, r0, f0);
        tmem_wait_ld32(r1);
        tmem_ld32_async(src + 64, r0);
        add32<16>(acc0, r1, f0);
        tmem_wait_ld32(r0);
        tmem_ld32_async(src + 96, r1);
        add32<0>(acc1, r0, f1);
        tmem_wait_ld32(r1);
        tc_fence_before();
        __syncwarp();
        if (elect_one()) mbar_arrive_pair(tempty + 16 * buf);
        add32<16>(acc1, r1, f1);
        if (kb % kScaleGroup == kScaleGroup - 1 || kb + 1 == a.k_blocks) {
          __syncwarp();
          if (elect_one()) mbar_arrive(bars.sempty(ring));
          ++group;
        }
      }
      if (!ok) break;
      // The tile is looked up and the thread asked for its place here, not before:
      // none of it occupies registers while the sums do.
      const Tile t = find(a, prefix, idx);
      const int tid = thread_index(), lane = tid & 31, quad = (tid >> 5) & 3, part = (tid >> 7) - 1;
      const int m0 = t.tok0 + rank * kHalf + quad * 32, n0 = t.row_block * kTileCol + part * 64;
      const uint32_t staging = sbase + kOffStaging + ((tid >> 5) - 4) * kStaging;
      store_tile<128, 2, 0, kFp32, kVec>(a, &tm_out, staging, m0, t.tok_end, n0, lane, acc0);
      store_tile<128, 2, 1, kFp32, kVec>(a, &tm_out, staging, m0, t.tok_end, n0 + kHalf, lane, acc1);
    }
    if (kVec && lane == 0) bulk_wait();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every product is read and no remote arrival is left
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem, kBufs * kHalf);
  cluster_sync();
}

}  // namespace paired

// ------------------------------------------------------------------ host side

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Rows of k bytes with a row pitch of ld bytes, read as 128-byte x box_rows
// boxes in the 128-byte swizzle; bytes past k and rows past the end read as 0.
static bool make_map(CUtensorMap* map, const void* p, int64_t k, int64_t rows, int64_t ld, int box_rows,
                     int box_bytes = kBlockK) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {(cuuint32_t)box_bytes, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The results' map for the stores of 32-row boxes; unused (zeros) where !kVec.
template <bool kFp32, bool kVec>
static bool make_out_map(CUtensorMap* map, const Args& a, int box_bytes) {
  constexpr int64_t kElt = kFp32 ? 4 : 2;
  if (kVec) return make_map(map, a.out, a.n * kElt, a.m, a.ldo * kElt, 32, box_bytes);
  *map = CUtensorMap{};
  return true;
}

// Token tiles of TN rows: at most this many exist, whatever the offsets say.
static int64_t most_token_tiles(const Args& a, int tn) {
  return a.offsets ? (int64_t)a.m / tn + std::min(a.experts, a.m) : ((int64_t)a.m + tn - 1) / tn;
}

// Stands in for gemm_kernel in the occupancy query, which answers one CTA per SM
// for any kernel that allocates TMEM (two are resident, by their columns and in
// fact): same threads and shared memory, no TMEM.
template <int kThreads, int kCtasPerSm>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) places_kernel() {}

// One kernel form on one device: its attributes, and how many clusters of 2, 4
// and 8 CTAs the device holds at once (GPCs of unequal size hold fewer than the
// SM count suggests).
template <int TN, bool kSplit, bool kFp32>
struct Form {
  using C = Cfg<TN, kSplit>;
  static constexpr auto kKernel = gemm_kernel<TN, kSplit, kFp32>;

  static void config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int64_t grid, int cluster,
                     cudaStream_t stream) {
    *cfg = cudaLaunchConfig_t{};
    cfg->gridDim = dim3((unsigned)grid);
    cfg->blockDim = dim3(C::kThreads);
    cfg->dynamicSmemBytes = C::kSmem;
    cfg->stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = cluster > 1 ? 2 : 1;
  }
  // clusters of `size` (2, 4, 8) CTAs that run at once on the device; 0 when unknown
  static int active_clusters(int device, int size) {
    static OncePerDevice once;
    static int count[kMaxDevices][3];
    const cudaError_t e = once.run(device, [&] {
      constexpr auto kPlaces = places_kernel<C::kThreads, C::kCtasPerSm>;
      cudaError_t err = cudaFuncSetAttribute(kPlaces, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      for (int i = 0; i < 3 && err == cudaSuccess; ++i) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        config(&cfg, attr, 2 << i, 2 << i, nullptr);
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
        err = cudaOccupancyMaxActiveClusters(&count[device][i], kPlaces, &cfg);
      }
      return err;
    });
    if (e != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    return count[device][size == 2 ? 0 : size == 4 ? 1 : 2];
  }
  static cudaError_t launch(const CUtensorMap& tm_w, const CUtensorMap& tm_a, const Args& a, int64_t grid, int device,
                            cudaStream_t stream) {
    static OncePerDevice once;
    const cudaError_t e = once.run(
        device, [] { return cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    config(&cfg, attr, grid, a.splits, stream);
    return cudaLaunchKernelEx(&cfg, kKernel, tm_w, tm_a, a);
  }
};

template <int TN, bool kFp32>
static cudaError_t launch_tn(const void* act, int64_t lda, const void* w, int64_t ldw, int64_t k, Args a, int splits,
                             Device dev, cudaStream_t stream) {
  using Split = Form<TN, true, kFp32>;
  using Whole = Form<TN, false, kFp32>;
  CUtensorMap tm_w, tm_a;
  if (!make_map(&tm_w, w, k, (int64_t)a.experts * a.n, ldw, kTileRows) || !make_map(&tm_a, act, k, a.m, lda, TN))
    return cudaErrorNotSupported;
  a.splits = splits;
  const int64_t tiles = most_token_tiles(a, TN) * a.row_blocks;
  if (splits > 1) return Split::launch(tm_w, tm_a, a, tiles * splits, dev.id, stream);
  return Whole::launch(tm_w, tm_a, a, std::min<int64_t>(tiles, (int64_t)dev.sms * Whole::C::kCtasPerSm), dev.id, stream);
}

template <bool kFp32, bool kVec>
static cudaError_t launch_square(const void* act, int64_t lda, const void* w, int64_t ldw, int64_t k, const Args& a,
                                 Device dev, cudaStream_t stream) {
  constexpr auto kernel = square::gemm_square_kernel<kFp32, kVec>;
  static OncePerDevice once;
  const cudaError_t e = once.run(
      dev.id, [] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, square::kSmem); });
  if (e != cudaSuccess) return e;
  CUtensorMap tm_w, tm_a, tm_out;
  if (!make_map(&tm_w, w, k, (int64_t)a.experts * a.n, ldw, square::kTileCol) ||
      !make_map(&tm_a, act, k, a.m, lda, square::kTileTok))
    return cudaErrorNotSupported;
  if (!make_out_map<kFp32, kVec>(&tm_out, a, 64)) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(most_token_tiles(a, square::kTileTok) * a.row_blocks, dev.sms));
  cfg.blockDim = dim3(square::kThreads);
  cfg.dynamicSmemBytes = square::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_a, tm_out, a);
}

template <bool kFp32, bool kVec>
static cudaError_t launch_paired(const void* act, int64_t lda, const void* w, int64_t ldw, int64_t k, Args a, Device dev,
                                 cudaStream_t stream) {
  constexpr auto kernel = paired::gemm_paired_kernel<kFp32, kVec>;
  static OncePerDevice once;
  const cudaError_t e = once.run(
      dev.id, [] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, paired::kSmem); });
  if (e != cudaSuccess) return e;
  CUtensorMap tm_w, tm_a, tm_out;
  if (!make_map(&tm_w, w, k, (int64_t)a.experts * a.n, ldw, paired::kHalf) ||
      !make_map(&tm_a, act, k, a.m, lda, paired::kHalf))
    return cudaErrorNotSupported;
  if (!make_out_map<kFp32, kVec>(&tm_out, a, 128)) return cudaErrorNotSupported;
  a.row_blocks = (a.n + paired::kTileCol - 1) / paired::kTileCol;
  const int64_t pairs = std::min<int64_t>(most_token_tiles(a, paired::kTileTok) * a.row_blocks, dev.sms / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(paired::kThreads);
  cfg.dynamicSmemBytes = paired::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_a, tm_out, a);
}

// The form with the least estimated time.  The estimate's constants are times in
// us, fitted to 640 timings on one GB300 (152 SMs; 1 to 8192 tokens, k 512 to
// 16384, every form), for the large tiles before their results left by TMA:
//   a k block of a swapped tile takes a CTA `alone` while it has its SM to itself
//   and `shared` of the SM's time when two CTAs share it;
//   the results of a tile cost `tile` more, the exchange of split sums `exchange`,
//   the launch and the first loads `fixed`;
//   the weights cannot come faster than 6.3 TB/s.
// On the present kernels the chosen form is the fastest one within 1.8 % on average
// over 90 dense sizes, 22 % at worst; grouped, with rows spread over all experts, 1 % and
// 3 %; with all rows on an eighth of the experts 10 % and 28 %, since every expert's
// weights are counted.  Where forms meet (n = k = 4096): 64 tokens 32 swapped in 4 parts
// 9.2, 64 in 4 9.7; 128 tokens 64 in 4 12.2, square 12.8; 512 tokens square 13.3,
// paired 20.2; 1024 tokens square 22.7, paired 20.9; 4096 tokens square 70.3, paired 66.9.
enum Shape { kSwapped16 = 16, kSwapped32 = 32, kSwapped64 = 64, kSquare = 128, kPaired = 256 };
struct Choice {
  double time = 1e30;
  int shape = kSwapped16, splits = 1;
  void offer(double t, int s, int parts) {
    if (t < time) {
      time = t;
      shape = s;
      splits = parts;
    }
  }
};

struct Cost {
  double alone, shared, tile, fixed, exchange;
};

// Tiles to expect.  Grouped rows: about half a tile of each expert is empty, and
// no tile serves two.
static int64_t expected_tiles(const Args& a, int tokens, int64_t row_tiles) {
  const int owners = std::min(a.experts, a.m);
  const double tok_tiles = a.offsets ? std::max((double)owners, (double)a.m / tokens + 0.5 * owners)
                                     : (double)most_token_tiles(a, tokens);
  return std::max<int64_t>(1, (int64_t)(tok_tiles * row_tiles));
}

// `clusters`: how many clusters of 2, 4 and 8 CTAs run at once (nullptr: asked of the device).
template <int TN, bool kFp32>
static void consider(const Args& a, Device dev, const int32_t* clusters, Cost c, double weights, Choice* choice) {
  constexpr int kPerSm = Cfg<TN, true>::kCtasPerSm;
  const int sms = dev.sms;
  const int64_t tiles = expected_tiles(a, TN, a.row_blocks), most = most_token_tiles(a, TN) * a.row_blocks;
  for (int i = 0, s = 1; s <= 8; ++i, s *= 2) {
    if (s > 1) {
      // every cluster runs at once, and a CTA keeps two blocks
      if (a.k_blocks < 2 * s || most * s > (int64_t)sms * kPerSm) break;
      if (most > (clusters ? clusters[i - 1] : Form<TN, true, kFp32>::active_clusters(dev.id, s))) break;
    }
    const int64_t on_sm = (tiles * s + sms - 1) / sms;  // CTAs of an SM, at once or one after the other
    const double chain = on_sm * (((a.k_blocks + s - 1) / s) * (on_sm == 1 ? c.alone : c.shared) + c.tile);
    choice->offer(std::max(chain, weights) + c.fixed + (s > 1 ? c.exchange : 0.0), TN, s);
  }
}

template <bool kFp32>
static Choice choose(const Args& a, Device dev, const int32_t* clusters) {
  Choice c;
  const int sms = dev.sms;
  const double weights = (double)std::min(a.experts, a.m) * a.n * a.k_blocks * kBlockK / 6.3e6;
  consider<16, kFp32>(a, dev, clusters, {0.244, 0.178, 0.5, 2.5, 1.2}, weights, &c);
  if (a.m > 16) consider<32, kFp32>(a, dev, clusters, {0.276, 0.191, 0.8, 2.4, 1.8}, weights, &c);
  if (a.m > 32) consider<64, kFp32>(a, dev, clusters, {0.395, 0.285, 1.4, 2.7, 2.2}, weights, &c);
  if (a.m > 64) {
    const int64_t rounds = (expected_tiles(a, square::kTileTok, a.row_blocks) + sms - 1) / sms;
    c.offer(std::max(rounds * (a.k_blocks * 0.253 + 1.4), weights) + 2.6, kSquare, 1);
  }
  if (a.m > 128) {
    const int64_t row_tiles = (a.n + paired::kTileCol - 1) / paired::kTileCol;
    const int64_t rounds = (expected_tiles(a, paired::kTileTok, row_tiles) + sms / 2 - 1) / (sms / 2);
    c.offer(std::max(rounds * (a.k_blocks * 0.45 + 1.0), weights) + 3.3, kPaired, 1);
  }
  return c;
}

// Whether the copy engine can store the results: 16-byte rows, a row pitch of
// fewer than 40 bits, and byte offsets within a row that its 32-bit coordinates hold.
template <bool kFp32>
static bool copied_results(const Args& a) {
  constexpr int64_t kElt = kFp32 ? 4 : 2;
  return a.ldo < (INT64_C(1) << 40) / kElt && a.ldo * kElt % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
         a.n * kElt <= INT32_MAX;
}

template <bool kFp32>
static cudaError_t launch_out(const void* act, int64_t lda, const void* w, int64_t ldw, int64_t k, const Args& a,
                              const GemmForm* form, Device dev, cudaStream_t stream) {
  Choice c;
  if (form) {
    c.shape = form->tile_tokens;
    c.splits = form->k_parts;
  } else {
    c = choose<kFp32>(a, dev, nullptr);
  }
  const bool vec = copied_results<kFp32>(a);
  switch (c.shape) {
    case kSwapped16: return launch_tn<16, kFp32>(act, lda, w, ldw, k, a, c.splits, dev, stream);
    case kSwapped32: return launch_tn<32, kFp32>(act, lda, w, ldw, k, a, c.splits, dev, stream);
    case kSwapped64: return launch_tn<64, kFp32>(act, lda, w, ldw, k, a, c.splits, dev, stream);
    case kSquare:
      return vec ? launch_square<kFp32, true>(act, lda, w, ldw, k, a, dev, stream)
                 : launch_square<kFp32, false>(act, lda, w, ldw, k, a, dev, stream);
  }
  return vec ? launch_paired<kFp32, true>(act, lda, w, ldw, k, a, dev, stream)
             : launch_paired<kFp32, false>(act, lda, w, ldw, k, a, dev, stream);
}

}  // namespace gemm8

static gemm8::Args gemm_args(const float* a_scales, int64_t a_scale_stride, const float* w_scales, const int32_t* offsets,
                             int m, int n, int k, int experts, void* out, int64_t ldo) {
  gemm8::Args a;
  a.a_scales = a_scales;
  a.w_scales = w_scales;
  a.offsets = offsets;
  a.out = out;
  a.a_scale_stride = a_scale_stride;
  a.ldo = ldo;
  a.m = m;
  a.n = n;
  a.k_blocks = (k + gemm8::kBlockK - 1) / gemm8::kBlockK;
  a.row_blocks = (n + gemm8::kTileRows - 1) / gemm8::kTileRows;
  a.scale_rows = a.row_blocks;
  a.experts = experts;
  a.splits = 1;
  a.give_up = -1;
  return a;
}

// The form that launch_gemm_fp8 chooses (`grouped`: offsets are given), and
// whether the copy engine stores its results.
void gemm_fp8_form(bool grouped, int m, int n, int k, int experts, const void* out, bool fp32, int64_t ldo, Device dev,
                   const int32_t* clusters, int* tile_tokens, int* k_parts, int* copied) {
  static const int32_t some = 0;  // not read
  const gemm8::Args a =
      gemm_args(nullptr, 0, nullptr, grouped ? &some : nullptr, m, n, k, experts, const_cast<void*>(out), ldo);
  const gemm8::Choice c = fp32 ? gemm8::choose<true>(a, dev, clusters) : gemm8::choose<false>(a, dev, clusters);
  *tile_tokens = c.shape;
  *k_parts = c.splits;
  *copied = c.shape >= gemm8::kSquare && (fp32 ? gemm8::copied_results<true>(a) : gemm8::copied_results<false>(a));
}

// Arguments are checked by the caller; cudaErrorNotSupported: the tensor-map
// encoder is unavailable or rejected the operands.  form: nullptr = the one
// with the least estimated time.
cudaError_t launch_gemm_fp8(const void* act, const float* a_scales, int64_t lda, int64_t a_scale_stride, const void* w,
                            const float* w_scales, int64_t ldw, const int32_t* offsets, int m, int n, int k,
                            int experts, void* out, bool fp32, int64_t ldo, const GemmForm* form, Device dev,
                            cudaStream_t stream) {
  gemm8::Args a = gemm_args(a_scales, a_scale_stride, w_scales, offsets, m, n, k, experts, out, ldo);
  if (form) a.give_up = form->give_up_warp;
  return fp32 ? gemm8::launch_out<true>(act, lda, w, ldw, k, a, form, dev, stream)
              : gemm8::launch_out<false>(act, lda, w, ldw, k, a, form, dev, stream);
}

cudaError_t gemm_read_error(int* code, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(code, gemm8::g_gemm_error, sizeof(int));
  if (e != cudaSuccess || !reset) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(gemm8::g_gemm_error, &zero, sizeof(int));
}

}  // namespace mla
