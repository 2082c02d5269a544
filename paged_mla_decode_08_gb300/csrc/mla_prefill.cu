// Latent attention in its expanded form, for prompts: every head has its own
// 128-wide keys and values, and the 64 rotary key columns are one row shared by
// all heads (sglang trtllm_mla_backend.py, forward_extend: ragged attention of
// head dims 192 / 128 with lse; tokenspeed trtllm_mla.py, TRTLLMMLABackend).
//
//   s_j = scale (q_nope . k_nope_j + q_pe . k_pe_j),   out = softmax(s) V,   lse = ln sum e^s
//
// One item: 512 query rows of one request and head on a pair of CTAs
// (cta_group::2), or 256 on one CTA; two tiles whose products and softmax
// alternate, each with 128 rows in every CTA.  A step is 128 keys (64 on one CTA):
//   S = Q K^T    (M = 128, N = 128, K = 192 a CTA)  operands in shared memory -> TMEM
//   P = 2^(c S - m) in registers, bf16, written over S
//   O += P V     (M = 128, N = 128, K = 128 a CTA)  P from TMEM, V from shared memory
// A thread of the softmax owns one query row, so its maximum and sum need no
// exchange.  While one tile's softmax runs, the tensor core has the other
// tile's products.  The running maximum only moves when a score exceeds it by
// 2^8 (P stays below 256, which bf16 and the fp32 sums hold); then that warp
// rescales its rows of O, which no product uses at that time: the products of a
// tile run in order, so S(j) in TMEM means that P V (j - 1) is done.  An item whose rows
// fill one tile or less has them in both, each with every second step ("alone"); the
// epilogue joins the two sums.
//
// Why pairs.  Q takes 96 KB of a CTA's shared memory.  One CTA reads 80 KB of keys
// and values a 128 keys, twice what the rest of its memory can hold ahead, and its
// products read 128 bytes of shared memory a cycle, all there is.  A pair's CTAs hold
// half of the keys and half of the value columns each: half the loads, half the reads
// of B, and three steps ahead.  19 heads, 2048 rows over 8192 keys: 108 us, 1880
// TFLOP/s (one CTA per 256 rows: 220 us).  One CTA an item has finer steps, rows and
// keys, for short requests.
//
// What bounds it.  Long prompts: the tensor core.  8192 tokens of 128 heads, causal: 1460
// to 1580 us (the products' floor at a library's burst rate is 1460), 1650 us in a
// loop of seconds under the power cap (98% of a library product's rate there).  Few rows
// over many keys: the bytes of keys and values; 8 requests of a row over 1000 to 4500 keys,
// 128 heads: 241 to 246 us, 5.9 TB/s.  Between them, what an item takes beside its steps: the
// first scores, the last weights' products and the epilogue come one after the other
// (a request of 130 tokens, 16 heads: 9 us with the launch, of which the data's
// floor is 0.4).
//
// P enters the second product in bf16 (half a step: 2^-8 of each weight at most, of
// random sign, below the rounding of the bf16 output); row sums and lse use the
// unrounded values.
//
// TMEM (512 columns): S / P of both tiles [0, 256), O of both tiles [256, 512).
// Shared memory: Q (2 x 48 KB) and a ring of three steps of 40 KB: 64 keys x 192
// columns, and 16 KB of values, in boxes of 64 columns in the 128-byte swizzle.
//
// Masked places.  Scores past a row's last key are replaced by -inf, so keys
// there may hold anything.  Values there are multiplied by P = 0, which leaves
// NaN of an infinity or a NaN; so the value tiles that some row does not see whole
// are looked through before they are used, and zeros put in the place of what is not
// finite.  The rows that do see such a value get it in the epilogue.
//
// Few row blocks and many keys: the keys of a block are cut into parts, each an item of
// its own, whose results in fp32 a second kernel merges.
//
// Warps: 0 TMA, 1 MMA, 2 none, 3 items, 4-7 softmax of the first tile,
// 8-11 of the second.  Waits are bounded: on timeout the error word is set, every role
// stops, copies and products in flight are awaited, TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <algorithm>
#include <mutex>

#include "../../include/mla_decode.h"
#include "mla_internal.h"
#include "mla_prompt.h"
#include "per_device.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace prefill {

using namespace mla::ptx;

__device__ int g_prefill_error;

constexpr int kRows = 128;               // query rows of a tile in a CTA
constexpr int kStages = 3;
constexpr int kBox = 64 * 128;           // 64 keys x 64 columns
constexpr int kQTile = 3 * 2 * kBox;     // 128 rows x 192 columns
constexpr int kKBytes = 3 * kBox;        // 64 keys x 192 columns of keys
constexpr int kVBytes = 2 * kBox;        // 64 keys x 128 or 128 keys x 64 columns of values
constexpr int kStageBytes = kKBytes + kVBytes;
constexpr int kOffQ = 0;
constexpr int kOffRing = 2 * kQTile;
constexpr int kOffBars = kOffRing + kStages * kStageBytes;
constexpr int kThreads = 384;
constexpr int kRegsLoad = 56, kRegsSoftmax = 224;  // 128 x 56 + 256 x 224 = 384 x 168, the launch's registers
constexpr float kRescaleLog2 = 8.0f;
constexpr long long kTimeoutCycles = 2000000000LL;

// kCtas: CTAs that share an item's keys
template <int kCtas>
struct Form {
  static constexpr int kKeys = 64 * kCtas;             // keys of a step
  static constexpr int kTileRows = kRows * kCtas;      // query rows of a tile
  static constexpr int kItemRows = 2 * kTileRows;
};

constexpr int kPartKeys = 256;  // of a part, at least
constexpr int kItemSlots = 4;
// Steps whose values are looked through: an item has at most five (its rows span four
// steps of keys), and a tile's warps, which may have nothing to do in an item, are at most
// kItemSlots items ahead of the other tile's.  With a barrier for each of those, the one
// that a warp comes to is behind in no phase, so a wait for either parity is not passed
// early.
constexpr int kLookBars = 32;
static_assert(kLookBars >= 5 * kItemSlots && kLookBars == 32, "every step in flight has its own; a lane sets one up");
constexpr int kAskAhead = 4;  // steps before an item's end at which its successor is asked for
enum Bar : int {
  B_Q = 0,                        // [tile] Q landed (the leader's barrier)
  B_QE = B_Q + 2,                 // [tile] Q is read
  B_KF = B_QE + 2,                // [stage] keys landed (the leader's)
  B_KE = B_KF + kStages,          // [stage] keys are read
  B_VF = B_KE + kStages,          // [stage] values landed (the leader's); not those to be looked through
  B_VE = B_VF + kStages,          // [stage] values are read
  B_RAW = B_VE + kStages,         // [look % kLookBars] values to be looked through landed
  B_S = B_RAW + kLookBars,        // [tile] scores are in TMEM
  B_P = B_S + 2,                  // [2 tile + half] weights are in TMEM, O is rescaled (the leader's)
  B_O = B_P + 4,                  // [tile] the tile's products are done
  B_ITEM = B_O + 2,               // [slot] an item is there
  B_TAKEN = B_ITEM + kItemSlots,  // [slot] every role of the item's CTAs has it (the leader's)
  B_STAT = B_TAKEN + kItemSlots,  // alone: the second tile's sums are there
  B_READ,                         // ... and its part of the output is read
  B_NEXT,                         // the item's copies come to their end: time to ask for the next
  B_ASKED,                        // the answer is there
  B_FIN,                          // every product is done
  B_COUNT
};
constexpr int kOffTmem = kOffBars + B_COUNT * 8;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kPoisons = 8;
constexpr int kOffPoison = kOffAbort + 4;
constexpr int kOffItem = (kOffPoison + 4 * kPoisons + 15) / 16 * 16;
constexpr int kOffAnswer = kOffItem + kItemSlots * 64;
constexpr int kOffStat = kOffAnswer + 16;  // [row] base and sum of the second tile
constexpr int kOffFirst = kOffStat + kRows * 8;  // the first 32 requests: offsets, then counts
constexpr int kSmem = kOffFirst + 32 * 32 + 1024;  // + alignment slack
static_assert(kSmem <= 232448, "shared memory budget");

constexpr uint32_t TM_S = 0, TM_O = 256, kTmemCols = 512;

struct Args {
  const int32_t* cu_q;
  const int32_t* cu_k;
  const uint16_t* v;
  uint16_t* out;
  float* lse;
  int64_t v_ts, v_hs, out_ts, out_hs;  // strides of a token and a head, in elements
  int32_t batch, heads, tokens_q, tokens_k;
  int32_t tiles;   // row blocks: at most this many exist
  int32_t parts;   // of a row block's keys, at most: each is an item of its own
  int32_t slots;   // CTAs, or pairs, that the GPU has room for
  int32_t group;   // heads whose items are mixed
  float* part_out; // [part][token][head][128], [part][token][head]: what a part alone gives
  float* part_lse;
  int32_t causal;
  float scale_log2;  // scale * log2(e)
};

// An item, as the scheduler hands it out (four 16-byte pieces).
struct Item {
  int q0, lq, k0, lk;   // the request's rows and keys
  int head, row0;       // first query row of the item within the request
  int part;             // of the keys' steps
  int more;             // 0: there is no item, the work is done
  // what it computes
  int begin;            // first step, in the request's keys; the others count from it
  int steps;
  int look;             // first step whose values are looked through: some row does not see it whole
  int alone;            // one tile's rows: the other tile takes them too, and every second step
  int tile_steps[2];    // a tile's share: the steps with a key that a row of it sees
  int end;              // behind the item's last row within the request
  int parts;            // of its keys
};
constexpr int kItemBytes = sizeof(Item);
static_assert(kItemBytes == 64, "pieces of an item");

__device__ __forceinline__ int visible(const Item& it, int causal, int row) {
  return causal ? max(0, min(it.lk, it.lk - it.lq + 1 + row)) : it.lk;
}
template <int kCtas>
__device__ __forceinline__ void plan_item(Item* it, const Args& a) {
  using F = Form<kCtas>;
  int all[2], total = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = it->row0 + t * F::kTileRows, last = min(first + F::kTileRows, it->end) - 1;
    all[t] = last >= first ? (visible(*it, a.causal, last) + F::kKeys - 1) / F::kKeys : 0;
    total = max(total, all[t]);
  }
  it->begin = 0;
  int end = total;
  if (it->parts > 1) {
    it->begin = total * it->part / it->parts;  // (fewer than 2^25 steps, at most 32 parts)
    end = total * (it->part + 1) / it->parts;
  }
  it->steps = it->look = end - it->begin;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it->tile_steps[t] = max(0, min(all[t], end) - it->begin);
    if (it->tile_steps[t] > 0)
      it->look = min(it->look, max(0, visible(*it, a.causal, it->row0 + t * F::kTileRows) / F::kKeys - it->begin));
  }
  it->alone = it->end - it->row0 <= F::kTileRows && it->steps > 1;
  if (it->alone) {
    it->tile_steps[0] = (it->steps + 1) / 2;
    it->tile_steps[1] = it->steps / 2;
  }
}
// First row of a CTA's share of a tile, within the request.
template <int kCtas>
__device__ __forceinline__ int first_row(const Item& it, int t, int rank) {
  return it.row0 + (it.alone ? 0 : t * Form<kCtas>::kTileRows) + rank * kRows;
}

// Row blocks, or the parts of their keys, one after the other: requests own ceil(rows / kItemRows) each, in their order; a request's
// come with the most keys first.  A request's first block takes what its rows leave over,
// for those see the fewest keys (128 heads, causal: 1537 rows 111 us with the last one taking
// it, 100 so; 16 requests of 300 rows 179 and 156).  Up to 32 requests come with the most
// keys first (8 requests of a row over 1000 to 4500 keys, 128 heads, 257 and 241 us; 10 of 1
// to 900 rows over 20 to 4512 keys, 16 heads, 79 and 65).  A request whose offsets break the
// rules, by themselves or by beginning before an earlier one's end, owns none.  Found by
// a warp that walks over the offsets, 32 requests at a time.
struct Walk {
  int base = 0;    // the next 32 requests
  int blocks = 0;  // row blocks, or parts, of those before
  int end = 0;     // ... and the latest end of their rows
};
// A lane's request of the next 32, its row blocks (or parts), how many there are up to
// it, and the parts of a block.
struct Request {
  int q0, q1, k0, k1, blocks, upto, parts;
  bool bad_q, bad_k;
};
// Up to 32 requests: a request's keys are cut so that no part is twice as long as all
// keys and row blocks, spread evenly, would make them (4 requests of 64 rows, 32 heads, three
// over 500 keys and one over 8000, 88 us uncut, 50 so).  More requests: all alike.
template <int kItemRows, bool kCut>
__device__ __forceinline__ Request walk_on(const Args& a, int batch, Walk& w, int lane) {
  Request r{};
  const int b = w.base + lane;
  if (b < batch) {
    // plain loads: the kernel before may write them while this one is resident
    r.q0 = a.cu_q[b];
    r.q1 = a.cu_q[b + 1];
    r.k0 = a.cu_k[b];
    r.k1 = a.cu_k[b + 1];
  }
  int before = r.q1;  // the latest end of the requests before this one
#pragma unroll
  for (int d = 1; d < 32; d *= 2) before = max(before, __shfl_up_sync(0xffffffffu, before, d) * (lane >= d));
  const int last = max(w.end, __shfl_sync(0xffffffffu, before, 31));
  before = __shfl_up_sync(0xffffffffu, before, 1);
  before = max(w.end, lane ? before : 0);
  const bool ok_q = r.q0 >= before && r.q0 <= r.q1 && r.q1 <= a.tokens_q, ok_k = r.k0 >= 0 && r.k0 <= r.k1 && r.k1 <= a.tokens_k;
  r.bad_q = b < batch && !ok_q;
  r.bad_k = b < batch && !ok_k;
  r.blocks = b < batch && ok_q && ok_k ? (r.q1 - r.q0 + kItemRows - 1) / kItemRows : 0;
  int all;
  r.parts = a.parts;
  if (batch <= 32) {
    const int keys = r.blocks > 0 ? r.k1 - r.k0 : 0;
    if (a.parts > 1) {
      // each operation rounded by itself: both kernels come to the same numbers
      float load = __fmul_rn(static_cast<float>(r.blocks), static_cast<float>(keys));
#pragma unroll
      for (int d = 1; d < 32; d *= 2) load = __fadd_rn(load, __shfl_xor_sync(0xffffffffu, load, d));
      const float even = __fdiv_rn(__fmul_rn(load, static_cast<float>(a.heads)), static_cast<float>(a.slots));
      const float share = fmaxf(static_cast<float>(kPartKeys), even);
      r.parts = max(1, min(a.parts, static_cast<int>(__fdiv_rn(static_cast<float>(keys), share))));
    }
    if (kCut) r.blocks *= r.parts;
    all = r.upto = 0;
#pragma unroll 1
    for (int i = 0; i < batch; ++i) {
      const int other = __shfl_sync(0xffffffffu, keys, i), blocks = __shfl_sync(0xffffffffu, r.blocks, i);
      all += blocks;
      if (other > keys || (other == keys && i <= lane)) r.upto += blocks;
    }
  } else {
    if (kCut) r.blocks *= r.parts;
    r.upto = r.blocks;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) r.upto += __shfl_up_sync(0xffffffffu, r.upto, d) * (lane >= d);
    all = __shfl_sync(0xffffffffu, r.upto, 31);
  }
  r.upto += w.blocks;
  w = Walk{w.base + 32, w.blocks + all, last};
  return r;
}
// All of them, and the first 32 requests; `report`: offsets that break the rules go to the
// error word.
template <int kItemRows, bool kCut>
__device__ __forceinline__ int count_blocks(const Args& a, int batch, int lane, bool report, Request* first) {
  Walk w;
  *first = walk_on<kItemRows, kCut>(a, batch, w, lane);
  bool bad_q = first->bad_q, bad_k = first->bad_k;
  while (w.base < batch) {
    const Request r = walk_on<kItemRows, kCut>(a, batch, w, lane);
    bad_q |= r.bad_q;
    bad_k |= r.bad_k;
  }
  if (report && (bad_q || bad_k)) atomicCAS(&g_prefill_error, 0, bad_q ? 0xA01 : 0xA02);
  return w.blocks;
}
// Row block, or part, number `idx`, if it is one of these requests'.
template <int kItemRows, bool kCut>
__device__ __forceinline__ bool pick_block(const Request& r, int idx, Item* it) {
  const unsigned hit = __ballot_sync(0xffffffffu, r.upto > idx && r.upto - r.blocks <= idx);
  if (!hit) return false;
  const int src = __ffs(hit) - 1;
  it->q0 = __shfl_sync(0xffffffffu, r.q0, src);
  it->lq = __shfl_sync(0xffffffffu, r.q1, src) - it->q0;
  it->k0 = __shfl_sync(0xffffffffu, r.k0, src);
  it->lk = __shfl_sync(0xffffffffu, r.k1, src) - it->k0;
  it->parts = __shfl_sync(0xffffffffu, r.parts, src);
  int block = __shfl_sync(0xffffffffu, r.upto, src) - 1 - idx;  // of the request
  it->part = 0;
  if (kCut && it->parts > 1) {
    const int at = block;
    block = at / it->parts;
    it->part = at - block * it->parts;
  }
  it->end = it->lq - ((it->lq - 1) / kItemRows - block) * kItemRows;
  it->row0 = max(0, it->end - kItemRows);
  return true;
}
// Number `idx`; false: there is none.  The walk goes on from where the last one ended,
// if that is not too far.
template <int kItemRows, bool kCut>
__device__ __forceinline__ bool find_block(const Args& a, int batch, int idx, Walk& from, int lane, Item* it) {
  Walk w;
  if (from.blocks <= idx) w = from;
  while (w.base < batch) {
    from = w;
    if (pick_block<kItemRows, kCut>(walk_on<kItemRows, kCut>(a, batch, w, lane), idx, it)) return true;
  }
  return false;
}

__device__ __forceinline__ uint32_t flag_load(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void flag_store(uint32_t addr, uint32_t v) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The leader of a pair waits for what its peer did as well.
template <int kCtas>
struct Ctx {
  uint32_t sbase, leader;  // shared-memory windows of this CTA and (as a cluster address) of the leader
  int rank;
  __device__ __forceinline__ uint32_t leader_bar(int i) const { return leader + kOffBars + 8 * i; }
  __device__ __forceinline__ uint32_t bar(int i) const { return sbase + kOffBars + 8 * i; }
  // Bounded wait; false: gave up here or elsewhere in the CTA.
  __device__ __forceinline__ bool wait(int i, uint32_t parity, int code) const {
    const uint32_t b = bar(i);
    if (mbar_try_wait(b, parity)) return true;
    const long long t0 = clock64();
    while (true) {
      if (mbar_try_wait(b, parity)) return true;
      if (flag_load(sbase + kOffAbort)) return false;
      if (clock64() - t0 > kTimeoutCycles) {
        flag_store(sbase + kOffAbort, 1);
        atomicCAS(&g_prefill_error, 0, code);
        return false;
      }
    }
  }
  // Whether a phase is over, for a converged warp.
  __device__ __forceinline__ bool ready(int i, uint32_t parity) const {
    return __all_sync(0xffffffffu, mbar_test_wait(bar(i), parity));
  }
  // For the issuing warp: the first tries loop inside one statement and the verdict is
  // a vote, so the compiler sees no divergence.
  __device__ __forceinline__ bool wait_uniform(int i, uint32_t parity, int code) const {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
        "TRY:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 64;\n\t@q bra TRY;\n"
        "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar(i)), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
    return wait_warp(i, parity, code);
  }
  __device__ __forceinline__ bool wait_warp(int i, uint32_t parity, int code) const {
    return __all_sync(0xffffffffu, wait(i, parity, code));
  }
  // Wait at a role's end: limited, without a verdict.
  __device__ __forceinline__ void wait_limited(int i, uint32_t parity) const {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar(i), parity) && clock64() - t0 < kTimeoutCycles) {
    }
  }
};

// ------------------------------------------------------------------ items

// The pair's CTAs take items together.  The leader asks the hardware for the next
// one (a cluster of this grid that has not started, which then never does): work is
// handed out as it gets done, and a CTA goes on to its next item without a launch,
// with its first copies and products under the last one's epilogue.
__device__ __forceinline__ void ask_for_cluster(uint32_t answer, uint32_t bar) {
  fence_proxy_async_smem();  // the last answer is read
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
               "r"(bar)
               : "memory");
}
// The first CTA of the cluster that the answer gives, or -1.
__device__ __forceinline__ int read_answer(uint32_t answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(answer)
      : "memory");
  return got ? (int)x : -1;
}

// What there is to do, and where a cluster stands: item `index`, then every
// `clusters`-th after it, then those of the cluster that the hardware gives.
struct Work {
  int blocks;    // parts of row blocks
  int items;     // ... of all heads
  int clusters;  // of the grid
  int index;     // -1: nothing is left
  Walk walk;
};
template <int kCtas>
__device__ __forceinline__ Work work_of(const Args& a, int blocks) {
  return Work{blocks, blocks * a.heads, (int)gridDim.x / kCtas, (int)blockIdx.x / kCtas, Walk()};
}
// Item `index`, for a converged warp.  Items come a row block at a time, a request's last
// and longest first, for a group of heads whose keys and values stay in L2; then
// the next group's.
template <int kCtas>
__device__ __forceinline__ Item item_of(const Args& a, Work& w, int lane, int batch, const Request& first) {
  Item it{};
  const int of_group = a.group * w.blocks, group = w.index / of_group, rest = w.index - group * of_group;
  const int heads = min(a.group, a.heads - group * a.group);
  const int block = rest / heads;
  it.head = group * a.group + rest - block * heads;
  constexpr int kRowsOf = Form<kCtas>::kItemRows;
  it.more = pick_block<kRowsOf, true>(first, block, &it) || find_block<kRowsOf, true>(a, batch, block, w.walk, lane, &it);
  plan_item<kCtas>(&it, a);
  return it;
}

template <int kCtas>
__device__ __forceinline__ void put_item(const Ctx<kCtas>& c, int slot, const Item& it) {
  const uint32_t dst = c.sbase + kOffItem + slot * kItemBytes;
  st_shared_v4(dst, make_uint4(it.q0, it.lq, it.k0, it.lk));
  st_shared_v4(dst + 16, make_uint4(it.head, it.row0, it.part, it.more));
  st_shared_v4(dst + 32, make_uint4(it.begin, it.steps, it.look, it.alone));
  st_shared_v4(dst + 48, make_uint4(it.tile_steps[0], it.tile_steps[1], it.end, it.parts));
}

// The first 32 requests, kept for the items to come.
template <int kCtas>
__device__ __forceinline__ void put_requests(const Ctx<kCtas>& c, int lane, const Request& r) {
  st_shared_v4(c.sbase + kOffFirst + 16 * lane, make_uint4(r.q0, r.q1, r.k0, r.k1));
  st_shared_v4(c.sbase + kOffFirst + 512 + 16 * lane, make_uint4(r.blocks, r.upto, r.parts, 0));
}
template <int kCtas>
__device__ __forceinline__ Request get_requests(const Ctx<kCtas>& c, int lane) {
  const uint4 x = ld_shared_v4(c.sbase + kOffFirst + 16 * lane), y = ld_shared_v4(c.sbase + kOffFirst + 512 + 16 * lane);
  return Request{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, false, false};
}

// Run by a warp of the leader: finds items and hands them to both CTAs.
template <int kCtas>
__device__ void schedule(const Ctx<kCtas>& c, const Args& a, Work w, Item it, int lane) {
  const uint32_t peer_items = kCtas > 1 ? mapa(c.sbase + kOffItem, 1) : 0;
  const uint32_t peer_bars = kCtas > 1 ? mapa(c.bar(B_ITEM), 1) : 0;
  int asked = 0;
  // The next index; false: a wait gave up.
  auto ask = [&] {
    if (lane == 0) ask_for_cluster(c.sbase + kOffAnswer, c.bar(B_ASKED));
    __syncwarp();
    const uint32_t parity = asked++ & 1;
    if (!c.wait_warp(B_ASKED, parity, 0xA1A)) {
      c.wait_limited(B_ASKED, parity);  // it comes in a microsecond or so, whatever else went wrong
      return false;
    }
    const int cta = read_answer(c.sbase + kOffAnswer);
    w.index = cta < 0 ? -1 : cta / kCtas;
    return true;
  };
  for (int n = 0;; ++n) {
    bool known = n == 0;  // the first item, if there is one, is in its slot
    while (w.index >= w.items) {  // fewer items than clusters: on to the next one
      if (!ask()) return;
      known = false;
    }
    if (w.index < 0)
      it.more = 0;
    else if (!known)
      it = item_of<kCtas>(a, w, lane, a.batch, get_requests(c, lane));
    const int slot = n % kItemSlots;
    if (n >= kItemSlots && !c.wait_warp(B_TAKEN + slot, (n / kItemSlots + 1) & 1, 0xA1B)) return;
    if (lane == 0) {
      if (!known) put_item(c, slot, it);  // (a first item is there)
      if (kCtas > 1) {
        const uint32_t dst = peer_items + slot * kItemBytes, bar = peer_bars + 8 * slot;
        st_async_v4(dst, it.q0, it.lq, it.k0, it.lk, bar);
        st_async_v4(dst + 16, it.head, it.row0, it.part, it.more, bar);
        st_async_v4(dst + 32, it.begin, it.steps, it.look, it.alone, bar);
        st_async_v4(dst + 48, it.tile_steps[0], it.tile_steps[1], it.end, it.parts, bar);
      }
      mbar_arrive(c.bar(B_ITEM + slot));
    }
    __syncwarp();
    if (!it.more) return;
    if (!c.wait_warp(B_NEXT, n & 1, 0xA1C)) return;
    if (w.index < w.items - w.clusters)
      w.index += w.clusters;
    else if (!ask())
      return;
  }
}
// ... and by one of its peer, whose slots the leader fills.
template <int kCtas>
__device__ void receive(const Ctx<kCtas>& c, int lane) {
  for (int n = 0;; ++n) {
    const int slot = n % kItemSlots;
    if (lane == 0) mbar_arrive_expect_tx(c.bar(B_ITEM + slot), kItemBytes);
    __syncwarp();
    if (!c.wait_warp(B_ITEM + slot, (n / kItemSlots) & 1, 0xA1E)) return;
    if (flag_load(c.sbase + kOffItem + slot * kItemBytes + 28) == 0) return;
  }
}

// Arrive on a barrier of the leader.  (What it orders is in place by then: this CTA's
// TMEM behind the tcgen05 fence, its shared memory behind a proxy fence or read already;
// a release at cluster scope would wait for all of it again, a thousand cycles.)
template <int kCtas>
__device__ __forceinline__ void arrive_leader(const Ctx<kCtas>& c, int bar) {
  if (kCtas > 1)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(c.leader_bar(bar)) : "memory");
  else
    mbar_arrive(c.bar(bar));
}

// Item n, for a converged warp, while its slot is held.
template <int kCtas>
__device__ __forceinline__ Item read_item(const Ctx<kCtas>& c, int n) {
  const uint32_t src = c.sbase + kOffItem + n % kItemSlots * kItemBytes;
  const uint4 x = ld_shared_v4(src), y = ld_shared_v4(src + 16), z = ld_shared_v4(src + 32);
  const uint4 w = ld_shared_v4(src + 48);
  return Item{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w,
              (int)z.x, (int)z.y, (int)z.z, (int)z.w, {(int)w.x, (int)w.y}, (int)w.z, (int)w.w};
}
// Wait for item n; false: there is none, or a wait gave up.
template <int kCtas>
__device__ __forceinline__ bool await_item(const Ctx<kCtas>& c, int n) {
  const int slot = n % kItemSlots;
  if (!c.wait_warp(B_ITEM + slot, (n / kItemSlots) & 1, 0xA1F)) return false;
  return flag_load(c.sbase + kOffItem + slot * kItemBytes + 28) != 0;
}
// The warp has what it needs of item n.
template <int kCtas>
__device__ __forceinline__ void release_item(const Ctx<kCtas>& c, int n) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive_leader(c, B_TAKEN + n % kItemSlots);
}
template <int kCtas>
__device__ __forceinline__ bool take_item(const Ctx<kCtas>& c, int n, Item* it) {
  if (!await_item(c, n)) return false;
  *it = read_item(c, n);
  release_item(c, n);
  return true;
}

// A place in a ring: counts on through all items.
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

// Load a box into this CTA's shared memory, completing on a barrier of the leader.
template <int kCtas>
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  if (kCtas > 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// Announce this CTA's bytes on a barrier of the leader (cluster address).  It orders
// nothing; a release at cluster scope would take the producer a thousand cycles each.
__device__ __forceinline__ void announce(uint32_t cluster_bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes)
               : "memory");
}

struct Maps {
  CUtensorMap q_nope, q_pe, k_nope, k_pe, v;
};

// ------------------------------------------------------------------ TMA

// Every CTA loads its own rows of Q, its 64 of the step's keys, and its columns of
// the step's values.  Values that are to be looked through complete on barriers of this
// CTA instead of the leader's.
template <int kCtas>
__device__ void load_items(const Ctx<kCtas>& c, const Args& a, const Maps& m, int lane) {
  using F = Form<kCtas>;
  Ring<kStages> ring;
  Ring<kLookBars> raw;
  uint32_t qe[2] = {1, 1};  // parities of Q's release
  int loaded = 0;           // stages used so far
  bool ok = true;
  Item it;
  for (int n = 0; ok && take_item(c, n, &it); ++n) {
    auto load_q = [&](int t) {
      if (it.tile_steps[t] == 0) return true;
      if (!c.wait_warp(B_QE + t, qe[t], 0xA10)) return false;
      qe[t] ^= 1;
      if (lane == 0) {
        const uint32_t dst = c.sbase + kOffQ + t * kQTile, bar = c.leader_bar(B_Q + t);
        const int row = it.q0 + first_row<kCtas>(it, t, c.rank);
        announce(bar, kQTile);
        tma_3d<kCtas>(dst, &m.q_nope, bar, 0, it.head, row);
        tma_3d<kCtas>(dst + 2 * kBox, &m.q_nope, bar, 64, it.head, row);
        tma_3d<kCtas>(dst + 4 * kBox, &m.q_pe, bar, 0, it.head, row);
      }
      __syncwarp();
      return true;
    };
    ok = load_q(0);
    for (int j = 0; ok && j < it.steps; ++j, ring.next()) {
      const int stage = ring.slot;
      const uint32_t dst = c.sbase + kOffRing + stage * kStageBytes;
      const int row = it.k0 + (it.begin + j) * F::kKeys;
      if (!(ok = c.wait_warp(B_KE + stage, ring.phase ^ 1, 0xA11))) break;
      if (lane == 0) {
        const uint32_t bar = c.leader_bar(B_KF + stage);
        announce(bar, kKBytes);
        tma_3d<kCtas>(dst, &m.k_nope, bar, 0, it.head, row + 64 * c.rank);
        tma_3d<kCtas>(dst + kBox, &m.k_nope, bar, 64, it.head, row + 64 * c.rank);
        tma_3d<kCtas>(dst + 2 * kBox, &m.k_pe, bar, 0, 0, row + 64 * c.rank);
      }
      __syncwarp();
      if (j == 0 && !(ok = load_q(1))) break;
      if (j == max(0, it.steps - kAskAhead) && c.rank == 0 && lane == 0) mbar_arrive(c.bar(B_NEXT));
      if (!(ok = c.wait_warp(B_VE + stage, ring.phase ^ 1, 0xA12))) break;
      ++loaded;
      const bool look = j >= it.look;
      if (lane == 0) {
        const uint32_t bar = look ? c.bar(B_RAW + raw.slot) : c.leader_bar(B_VF + stage);
        if (look)
          mbar_arrive_expect_tx(bar, kVBytes);
        else
          announce(bar, kVBytes);
        tma_3d<kCtas>(dst + kKBytes, &m.v, bar, 64 * c.rank, it.head, row);
        if (kCtas == 1) tma_3d<kCtas>(dst + kKBytes + kBox, &m.v, bar, 64, it.head, row);
      }
      __syncwarp();
      if (look) raw.next();
    }
    if (ok && it.steps == 0 && c.rank == 0 && lane == 0) mbar_arrive(c.bar(B_NEXT));
    __syncwarp();
  }
  if (!ok) {  // the copies in flight land within a few microseconds
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) {
    }
  }
  // Every copy has landed, and every arrival that the products send here has come
  // in, before this CTA may leave.  (The products follow the copies.)
  for (int k = 0; k < kStages; ++k, ring.next()) {  // from the oldest stage on
    if (k < kStages - loaded) continue;             // never used
    c.wait_limited(B_KE + ring.slot, ring.phase ^ 1);
    c.wait_limited(B_VE + ring.slot, ring.phase ^ 1);
  }
}

// ------------------------------------------------------------------ MMA

// Operand descriptors differ in the start address alone (the low word).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (kSwizzle128B << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); }

// Four K = 16 products, D[tmem] (+)= A B^T, for a CTA or a pair: A in shared memory
// (`a` a low word, a step 32 bytes) or in TMEM (`a` an address, a step 8 columns), B
// in shared memory (a step 32 bytes of keys, or 16 keys of values).  The whole issuing
// warp runs through, one lane (`go`) issues: with predicated instructions and no
// divergence descriptors stay in uniform registers.  (One lane in a branch of its own
// took 95 to 120 cycles a product, which the tensor core does in 64.)
template <int kCtas>
__device__ __forceinline__ void products_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate,
                                            uint32_t go) {
  if (kCtas == 1)
    asm volatile(
        "{\n\t.reg .pred g, p;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\tsetp.ne.b32 g, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t@g tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 da, {x, %6};\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 da, {x, %6};\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 da, {x, %6};\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(go), "r"(kDescHigh)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred g, p;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\tsetp.ne.b32 g, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t@g tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 da, {x, %6};\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 da, {x, %6};\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 da, {x, %6};\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t"
        "}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(go), "r"(kDescHigh)
        : "memory");
}
template <int kCtas>
__device__ __forceinline__ void products_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate,
                                            uint32_t go) {
  if (kCtas == 1)
    asm volatile(
        "{\n\t.reg .pred g, p;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\tsetp.ne.b32 g, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %6};\n\t@g tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "add.u32 x, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 x, %1, 16;\n\tadd.u32 y, %2, 256;\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 x, %1, 24;\n\tadd.u32 y, %2, 384;\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(go), "r"(kDescHigh)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred g, p;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\tsetp.ne.b32 g, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %6};\n\t@g tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "add.u32 x, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::2.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 x, %1, 16;\n\tadd.u32 y, %2, 256;\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::2.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 x, %1, 24;\n\tadd.u32 y, %2, 384;\n\tmov.b64 db, {y, %6};\n\t@g tcgen05.mma.cta_group::2.kind::f16 [%0], [x], db, %3, p;\n\t"
        "}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(go), "r"(kDescHigh)
        : "memory");
}
// Arrive on the barrier at this offset in every CTA when the products issued so far are done.
template <int kCtas>
__device__ __forceinline__ void commit(uint32_t bar, uint32_t go) {
  if (kCtas == 1)
    asm volatile(
        "{\n\t.reg .pred g;\n\tsetp.ne.b32 g, %1, 0;\n\t"
        "@g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(go)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred g;\n\tsetp.ne.b32 g, %1, 0;\n\t"
        "@g tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(bar),
        "r"(go), "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}

// Run by a whole warp.  In turn: O += P V of a tile's last step and S = Q K^T of its
// next one, then the same of the other tile, on through all items.
template <int kCtas>
__device__ void issue_products(const Ctx<kCtas>& c, const Args& a, uint32_t tmem) {
  using F = Form<kCtas>;
  constexpr uint32_t kIdescS = idesc_f32acc(F::kTileRows, F::kKeys, 0, 0, 1);
  constexpr uint32_t kIdescO = idesc_f32acc(F::kTileRows, 128, 0, 1, 1);
  const uint32_t go = elect_one();
  const uint32_t q0 = desc_low(c.sbase + kOffQ, 16), k0 = desc_low(c.sbase + kOffRing, 16);
  const uint32_t v0 = desc_low(c.sbase + kOffRing + kKBytes, kBox);
  Ring<kStages> kr, vr;              // the next step's keys, the last step's values
  // of each tile a bit
  uint32_t qp = 0, pp = 0;           // parities of Q and of P
  uint32_t due = 0;                  // the last step's second product is still to come
  uint32_t first = 0, last = 0;      // ... of that step in its item
  uint32_t looked = 0;               // its values are looked through: with the weights comes the word that they can be used
  uint32_t vp = 0;                   // [stage] of the values that are not looked through
  bool alone = false, was_alone = false;  // the tiles have steps of their own: of the next, of the last step
  bool ok = true, more = true;
  Item it;
  for (int n = 0; ok && more;) {
    // What is still to come is not held up by an item that is not there yet.
    const bool take = !due || c.ready(B_ITEM + n % kItemSlots, (n / kItemSlots) & 1);
    if (take) more = take_item(c, n++, &it);
    const bool keys = take && more;
    const int steps0 = keys ? it.tile_steps[0] : 0, steps1 = keys ? it.tile_steps[1] : 0;
    const int total = keys ? max(steps0, steps1) : 1, look = it.look;
    if (keys) alone = it.alone;
    for (int j = 0; ok && j < total; ++j) {
      const uint32_t was = due;
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const uint32_t bit = 1u << t, d = tmem + TM_O + 128 * t, p = tmem + TM_S + 128 * t;
        if (was & bit) {
          if ((t == 0 || !(was & 1) || was_alone) && !(looked & bit)) {
            if (!(ok = c.wait_uniform(B_VF + vr.slot, (vp >> vr.slot) & 1, 0xA13))) break;
            vp ^= 1u << vr.slot;
          }
          const uint32_t v = v0 + vr.slot * (kStageBytes >> 4);
#pragma unroll
          for (int half = 0; half < kCtas; ++half) {  // 64 keys each; 64 value columns of a key are 128 bytes
            if (!(ok = c.wait_uniform(B_P + 2 * t + half, (pp >> t) & 1, 0xA14))) break;
            tc_fence_after();
            products_ts<kCtas>(d, p + 32 * half, v + 512 * half, kIdescO, !(first & bit) || half > 0, go);
          }
          if (!ok) break;
          pp ^= bit;
          if (last & bit) commit<kCtas>(c.bar(B_O + t), go);
          if (t == 1 || !(was & 2) || was_alone) {  // its last reader
            commit<kCtas>(c.bar(B_VE + vr.slot), go);
            vr.next();
          }
          due &= ~bit;
        }
        const int steps = t ? steps1 : steps0;
        if (j < steps) {
          if ((t == 0 || j >= steps0 || alone) && !(ok = c.wait_uniform(B_KF + kr.slot, kr.phase, 0xA15))) break;
          if (j == 0) {
            if (!(ok = c.wait_uniform(B_Q + t, (qp >> t) & 1, 0xA16))) break;
            qp ^= bit;
          }
          tc_fence_after();
          const uint32_t q = q0 + t * (kQTile >> 4), k = k0 + kr.slot * (kStageBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 3; ++kk)
            products_ss<kCtas>(p, q + kk * (2 * kBox >> 4), k + kk * (kBox >> 4), kIdescS, kk > 0, go);
          commit<kCtas>(c.bar(B_S + t), go);
          if (j == steps - 1) commit<kCtas>(c.bar(B_QE + t), go);
          if (t == 1 || j >= steps1 || alone) {
            commit<kCtas>(c.bar(B_KE + kr.slot), go);
            kr.next();
          }
          due |= bit;
          first = (first & ~bit) | (j == 0 ? bit : 0);
          last = (last & ~bit) | (j == steps - 1 ? bit : 0);
          looked = (looked & ~bit) | ((alone ? 2 * j + t : j) >= look ? bit : 0);
        }
      }
      was_alone = alone;
    }
  }
  // every product is done before TMEM is released
  commit<kCtas>(c.bar(B_FIN), go);
  c.wait_limited(B_FIN, 0);
}

// ------------------------------------------------------------------ masked values

// Zeros in the place of what is not finite, in a quarter (32 keys, or 16 of two boxes)
// of this CTA's values of a step; `own`: keys of it that are the request's.  True: some
// of those were not finite.
template <int kCtas>
__device__ bool look_through(uint32_t values, int quarter, int lane, int own) {
  using F = Form<kCtas>;
  const uint32_t base = values + quarter * (kVBytes / 4) + lane * 16;
  constexpr uint32_t kExp = 0x7F807F80u, kOne = 0x00800080u, kTop = 0x80008000u;  // an exponent of ones carries into the sign
  uint4 x[8];
  uint32_t found = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = ld_shared_v4(base + i * 512);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    found |= ((x[i].x & kExp) + kOne) | ((x[i].y & kExp) + kOne) | ((x[i].z & kExp) + kOne) | ((x[i].w & kExp) + kOne);
  bool seen = false;
  if (found & kTop) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      uint4 y = ld_shared_v4(base + i * 512);
      const uint32_t b0 = __vcmpeq2(y.x & kExp, kExp), b1 = __vcmpeq2(y.y & kExp, kExp), b2 = __vcmpeq2(y.z & kExp, kExp),
                     b3 = __vcmpeq2(y.w & kExp, kExp);
      if (b0 | b1 | b2 | b3) {
        st_shared_v4(base + i * 512, make_uint4(y.x & ~b0, y.y & ~b1, y.z & ~b2, y.w & ~b3));
        // a key is 128 bytes; one CTA alone holds two boxes of 64 keys
        seen |= (quarter * 32 + i * 4 + (lane >> 3)) % F::kKeys < own;
      }
    }
    fence_proxy_async_smem();
  }
  return seen;
}

// ------------------------------------------------------------------ softmax

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
#define MLA_I8(b) "r"(r[b + 0]), "r"(r[b + 1]), "r"(r[b + 2]), "r"(r[b + 3]), "r"(r[b + 4]), "r"(r[b + 5]), \
                  "r"(r[b + 6]), "r"(r[b + 7])
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      MLA_I8(0), MLA_I8(8)
      : "memory");
}
#undef MLA_I8
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void store32(uint16_t* p, const uint32_t* r, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// Adds to a row's written results what is not finite among the values of keys [from, to),
// column by column: such a value weighs something, so an infinity or a NaN is what a
// row that sees it gets.
template <class T>
__device__ __noinline__ void add_non_finite(const uint16_t* v, int64_t stride, int from, int to, T* out) {
  for (int col = 0; col < 128; ++col) {
    float sum = 0.f;
    for (int key = from; key < to; ++key) {
      const uint32_t bits = v[key * stride + col];
      if ((bits & 0x7F80u) == 0x7F80u) sum += __uint_as_float(bits << 16);
    }
    if (sum == 0.f) continue;
    if constexpr (sizeof(T) == 2)
      out[col] = __float2bfloat16_rn(__bfloat162float(out[col]) + sum);
    else
      out[col] += sum;
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
union Pair {
  float2 f;
  uint64_t u;
};
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  Pair x, y, z, d;
  x.f = a; y.f = b; z.f = c;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.u) : "l"(x.u), "l"(y.u), "l"(z.u));
  return d.f;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  Pair x, y, d;
  x.f = a; y.f = b;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(x.u), "l"(y.u));
  return d.f;
}

// Weights 2^(c s - base) of 32 scores, packed, and their sum onto two pairs.
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], float2 scale, float base, uint32_t* p, float2 (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float2 x = fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale, make_float2(-base, -base));
    x.x = ex2_approx(x.x);
    x.y = ex2_approx(x.y);
    sum[i & 1] = add2(sum[i & 1], x);
    p[i] = pack(x.x, x.y);
  }
}
__device__ __forceinline__ void mask32(uint32_t (&s)[32], int left) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i >= left) s[i] = 0xFF800000u;  // -inf
}
__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
#pragma unroll
  for (int i = 2; i < 32; i += 4) {
    a = max3(a, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    if (i + 3 < 32) b = max3(b, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
  }
  return fmaxf(a, b);
}

// Item n has values of its own that are not finite: told to both CTAs, since each looks
// through half of the columns.
template <int kCtas>
__device__ __forceinline__ void note_non_finite(const Ctx<kCtas>& c, int n) {
  const uint32_t at = c.sbase + kOffPoison + 4 * (n % kPoisons);
  flag_store(at, 1);
  if (kCtas > 1) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa(at, c.rank ^ 1)), "r"(1) : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
  }
}

// A tile's first steps, of which every row of a CTA sees every key and no values are to
// be looked through.
template <int kCtas>
__device__ __forceinline__ int whole_steps(const Item& it, int causal, int t, int rank) {
  const int row = min(first_row<kCtas>(it, t, rank), it.end - 1);
  const int masked = visible(it, causal, row) / Form<kCtas>::kKeys - it.begin;
  const int some = min(masked, t == 0 || it.alone ? it.look : max(it.look, it.tile_steps[0]));
  const int mine = it.alone ? (some - t + 1) / 2 : some;  // of this tile's
  return min(t ? it.tile_steps[1] : it.tile_steps[0], max(0, mine));
}

// The softmax and the epilogue of one tile, for every item: four warps, a row a
// thread.  The weights of a step's first half are made with the running maximum as it
// was, while the step's own is found (the exponentials' pipe and the comparisons' run
// side by side); should it have to move, which is rare after the first step, they
// are made again.  The first half is handed to the tensor core before the second one
// is made.
template <int kCtas>
__device__ void softmax_items(const Ctx<kCtas>& c, const Args& a, int t, uint32_t tmem) {
  using F = Form<kCtas>;
  constexpr int kParts = F::kKeys / 32;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t ts = tmem + lanes + TM_S + 128 * t, to = tmem + lanes + TM_O + 128 * t;
  const float slack = kRescaleLog2 / a.scale_log2;
  const float2 scale = make_float2(a.scale_log2, a.scale_log2);
  uint32_t sp = 0, op = 0, other_op = 0, ap = 0;  // parities of S, O, the other tile's O, and what passes between them
  int vstep = 0, looks = 0;  // steps, and steps looked through, of the items before
  float top, base;           // the running maximum of S, and of c S (0 while there is none)
  float2 sum[2];
  // The running maximum moves to `here` where that is too far above it; `fresh`: there
  // is no output yet, which else is rescaled.
  auto move_to = [&](float here, bool fresh) {
    const bool up = here > top + slack;
    const float factor = up ? ex2_approx((top - here) * a.scale_log2) : 1.f;
    if (up) {
      top = here;
      base = here * a.scale_log2;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) sum[i] = make_float2(sum[i].x * factor, sum[i].y * factor);
    if (fresh) return;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      uint32_t o[32];
      tmem_ld32(to + 32 * q, o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
      tmem_st32(to + 32 * q, o);
    }
  };
  // The weights stored so far are in TMEM: hand them over.
  auto hand_over = [&](int half) {
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_leader(c, B_P + 2 * t + half);
  };
  // A step that every row sees whole.
  auto whole_step = [&](bool fresh) {
    if (!c.wait_warp(B_S + t, sp, 0xA18)) return false;
    sp ^= 1;
    tc_fence_after();
    constexpr int kHalf = kParts / 2;
    uint32_t s[kHalf][32], p[16 * kHalf];
    float here;
    {
      uint32_t u[kHalf][32];  // the second half, for the maximum
#pragma unroll
      for (int q = 0; q < kHalf; ++q) tmem_ld32_async(ts + 32 * q, s[q]);
#pragma unroll
      for (int q = 0; q < kHalf; ++q) tmem_ld32_async(ts + 32 * (kHalf + q), u[q]);
#pragma unroll
      for (int q = 0; q < kHalf; ++q) tmem_wait_ld32(s[q]);
#pragma unroll
      for (int q = 0; q < kHalf; ++q) tmem_wait_ld32(u[q]);
      here = fmaxf(max32(s[0]), max32(u[0]));
      if (kHalf == 2) here = max3(here, max32(s[kHalf - 1]), max32(u[kHalf - 1]));
    }
    float2 more[2] = {sum[0], sum[1]};
    if (!fresh) {
#pragma unroll
      for (int q = 0; q < kHalf; ++q) weights32(s[q], scale, base, p + 16 * q, more);
    }
    if (fresh || __any_sync(0xffffffffu, here > top + slack)) {
      move_to(here, fresh);
      more[0] = sum[0];
      more[1] = sum[1];
#pragma unroll
      for (int q = 0; q < kHalf; ++q) weights32(s[q], scale, base, p + 16 * q, more);
    }
#pragma unroll
    for (int q = 0; q < kHalf; ++q) tmem_st16_async(ts + 16 * q, p + 16 * q);
#pragma unroll
    for (int q = 0; q < kHalf; ++q) tmem_ld32_async(ts + 32 * (kHalf + q), s[q]);  // (P ends before)
    if (kCtas > 1) hand_over(0);
#pragma unroll
    for (int q = 0; q < kHalf; ++q) {
      tmem_wait_ld32(s[q]);
      weights32(s[q], scale, base, p + 16 * q, more);
      tmem_st16_async(ts + 16 * (kHalf + q), p + 16 * q);
    }
    sum[0] = more[0];
    sum[1] = more[1];
    hand_over(kCtas - 1);
    return true;
  };
  // A step of which this thread's row sees `left` keys, 32 at a time in loops: it comes a few
  // times an item, and what it costs is to fetch its instructions (unrolled it took
  // 3000 to 3500 cycles where a whole step takes 1400).
  auto edge_step = [&](bool fresh, int left) {
    if (!c.wait_warp(B_S + t, sp, 0xA18)) return false;
    sp ^= 1;
    tc_fence_after();
    const int most = __shfl_sync(0xffffffffu, left, 31);  // rows see more and more
    uint32_t s[32];
    float here = -CUDART_INF_F;
#pragma unroll 1
    for (int q = 0; q < kParts && 32 * q < most; ++q) {
      tmem_ld32(ts + 32 * q, s);
      mask32(s, left - 32 * q);
      here = fmaxf(here, max32(s));
    }
    if (fresh || __any_sync(0xffffffffu, here > top + slack)) move_to(here, fresh);
#pragma unroll 1
    for (int q = 0; q < kParts; ++q) {
      uint32_t p[16];
      if (32 * q < most) {
        tmem_ld32(ts + 32 * q, s);
        mask32(s, left - 32 * q);
        weights32(s, scale, base, p, sum);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = 0;
      }
      tmem_st16_async(ts + 16 * q, p);  // (over scores that are read)
      if (kCtas > 1 && q == kParts / 2 - 1) hand_over(0);
    }
    hand_over(kCtas - 1);
    return true;
  };
  for (int n = 0; await_item(c, n); ++n) {
    // Steps that every row sees whole need nothing of the item; what it is is read again
    // behind them, so that it takes no registers meanwhile.
    const int whole = whole_steps<kCtas>(read_item(c, n), a.causal, t, c.rank);
    top = -CUDART_INF_F;
    base = 0.f;
    sum[0] = sum[1] = make_float2(0.f, 0.f);
    for (int j = 0; j < whole; ++j)
      if (!whole_step(j == 0)) return;

    const Item it = read_item(c, n);
    const int mine_steps = t ? it.tile_steps[1] : it.tile_steps[0], other_steps = t ? it.tile_steps[0] : it.tile_steps[1];
    const int values = vstep, look0 = looks;
    vstep = (vstep + it.steps) % kStages;
    looks = (looks + it.steps - it.look) % (2 * kLookBars);
    if (t == 0 && quad == 0) flag_store(c.sbase + kOffPoison + 4 * ((n + kPoisons / 2) % kPoisons), 0);
    // A tile's steps are every one of the item's, or every second one.
    const int stride = it.alone ? 2 : 1, shift = it.alone ? t : 0;
    // The first active tile's warps look through a step's values, before its weights are handed over.
    const int looker = t == 0 || it.alone ? it.look : max(it.look, it.tile_steps[0]);
    auto look = [&](int j) {
      if (j < looker) return true;
      const int k = look0 + j - it.look;
      if (!c.wait_warp(B_RAW + k % kLookBars, (k / kLookBars) & 1, 0xA17)) return false;
      const uint32_t at = c.sbase + kOffRing + (values + j) % kStages * kStageBytes + kKBytes;
      if (look_through<kCtas>(at, quad, lane, it.lk - (it.begin + j) * F::kKeys))
        note_non_finite(c, n);
      return true;
    };
    const int row = first_row<kCtas>(it, t, c.rank) + quad * 32 + lane;  // within the request
    const int seen = visible(it, a.causal, min(row, it.end - 1));
    for (int i = whole; i < mine_steps; ++i) {
      const int j = i * stride + shift;
      if (!look(j) || !edge_step(i == 0, seen - (it.begin + j) * F::kKeys)) return;
    }
    // ---- epilogue
    float total = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y), mine_f = 1.f, other_f = 0.f;
    const uint32_t stat = c.sbase + kOffStat + (quad * 32 + lane) * 8;
    if (it.alone && t == 1) {
      // the first tile's warps write both tiles' rows
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(stat), "f"(base), "f"(total) : "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar(B_STAT));
      if (!c.wait_warp(B_READ, ap, 0xA20)) return;
      ap ^= 1;
      op ^= 1;
      other_op ^= 1;
      release_item(c, n);
      continue;
    }
    if (it.alone) {
      if (!c.wait_warp(B_STAT, ap, 0xA21)) return;
      ap ^= 1;
      float b, l;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(b), "=f"(l) : "r"(stat) : "memory");
      const float m = total == 0.f ? b : l == 0.f ? base : fmaxf(base, b);
      mine_f = total == 0.f ? 0.f : ex2_approx(base - m);
      other_f = l == 0.f ? 0.f : ex2_approx(b - m);
      base = m;
      total = total * mine_f + l * other_f;
    }
    const bool mine = row < it.end;
    const bool none = total == 0.f;  // no key, or scores of -inf alone
    // a share of no weight may hold anything
    const uint32_t keep = none || mine_f == 0.f ? 0 : ~0u, keep_other = none || other_f == 0.f ? 0 : ~0u;
    const float inv = __fdividef(mine_f, total), other_inv = __fdividef(other_f, total);
    const int64_t token = it.q0 + row, part_row = (int64_t)it.part * a.tokens_q + token;
    uint16_t* out = a.out + token * a.out_ts + it.head * a.out_hs;
    float* part_out = a.part_out + (part_row * a.heads + it.head) * 128;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    // The first turn reads and writes nothing: it has the loop's instructions fetched
    // while the last products run (900 cycles an item).
#pragma unroll 1
    for (int q = -1; q < 4; ++q) {
      if (q == 0 && mine_steps > 0) {
        if (!c.wait_warp(B_O + t, op, 0xA19) || (it.alone && !c.wait_warp(B_O + 1, other_op, 0xA1D))) return;
        tc_fence_after();
      }
      uint32_t r[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = 0;
      if (q >= 0 && mine_steps > 0) tmem_ld32(to + 32 * q, r);
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i] & keep) * inv);
      if (it.alone) {
        uint32_t u[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = 0;
        if (q >= 0) tmem_ld32(tmem + lanes + TM_O + 128 + 32 * q, u);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          r[i] = __float_as_uint(fmaf(__uint_as_float(u[i] & keep_other), other_inv, __uint_as_float(r[i])));
        if (q == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(c.bar(B_READ));
        }
      }
      if (it.parts > 1) {
        if (mine && !none && q >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            reinterpret_cast<uint4*>(part_out + 32 * q)[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
        continue;
      }
      uint32_t p[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      if (none) {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = 0;
      }
      if (mine && q >= 0) {
        store32(out + 32 * q, p, wide);
        store32(out + 32 * q + 16, p + 8, wide);
      }
    }
    if (mine_steps > 0) op ^= 1;
    if (other_steps > 0) other_op ^= 1;
    const bool poison = flag_load(c.sbase + kOffPoison + 4 * (n % kPoisons)) != 0;
    float* lse = it.parts > 1 ? a.part_lse + part_row * a.heads : a.lse + token * a.heads;
    if (poison && mine && !none) {
      const uint16_t* v = a.v + it.k0 * a.v_ts + it.head * a.v_hs;
      const int from = (it.begin + it.look) * F::kKeys, to = min(seen, (it.begin + it.steps) * F::kKeys);
      if (it.parts > 1)
        add_non_finite(v, a.v_ts, from, to, part_out);
      else
        add_non_finite(v, a.v_ts, from, to, reinterpret_cast<__nv_bfloat16*>(out));
    }
    release_item(c, n);
    if (mine) lse[it.head] = none ? -CUDART_INF_F : fmaf(base, CUDART_LN2_F, logf(total));
  }
}

template <int kCtas>
__device__ __forceinline__ void tmem_alloc_of(uint32_t dst) {
  if (kCtas == 1) {
    tmem_alloc(dst, kTmemCols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int kCtas>
__device__ __forceinline__ void tmem_dealloc_of(uint32_t tmem) {
  if (kCtas == 1)
    tmem_dealloc(tmem, kTmemCols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <int kCtas>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctx<kCtas> c;
  c.sbase = smem_u32(smem);
  c.rank = kCtas > 1 ? (int)cluster_ctarank() : 0;
  c.leader = kCtas > 1 ? mapa(c.sbase, 0) : c.sbase;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  int blocks = 0;
  Item own;
  if (warp == 3 && c.rank == 0) {
    // A first turn on nothing has the instructions fetched while the work before this
    // launch is not done.
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
      if (turn) asm volatile("griddepcontrol.wait;" ::: "memory");
      Request first;
      blocks = count_blocks<Form<kCtas>::kItemRows, true>(a, turn ? a.batch : 0, lane, blockIdx.x == 0, &first);
      Work work = work_of<kCtas>(a, turn ? blocks : 1);
      if (turn == 0 || work.index < work.items) own = item_of<kCtas>(a, work, lane, turn ? a.batch : 0, first);
      put_requests(c, lane, first);
      if (lane == 0) put_item(c, 0, own);
    }
  } else if (warp == 0) {
    mbar_init(c.bar(B_RAW + lane), 1);
    fence_mbar_init();
    if (lane == 0) {
      flag_store(c.sbase + kOffAbort, 0);
      for (int i = 0; i < kPoisons; ++i) flag_store(c.sbase + kOffPoison + 4 * i, 0);
      for (int t = 0; t < 2; ++t) {
        mbar_init(c.bar(B_Q + t), kCtas);
        mbar_init(c.bar(B_QE + t), 1);
        mbar_init(c.bar(B_S + t), 1);
        mbar_init(c.bar(B_P + 2 * t), 4 * kCtas);
        mbar_init(c.bar(B_P + 2 * t + 1), 4 * kCtas);
        mbar_init(c.bar(B_O + t), 1);
      }
      for (int i = 0; i < kStages; ++i) {
        mbar_init(c.bar(B_KF + i), kCtas);
        mbar_init(c.bar(B_KE + i), 1);
        mbar_init(c.bar(B_VF + i), kCtas);
        mbar_init(c.bar(B_VE + i), 1);
      }
      for (int i = 0; i < kItemSlots; ++i) {
        mbar_init(c.bar(B_ITEM + i), 1);
        mbar_init(c.bar(B_TAKEN + i), 9 * kCtas + 1);  // copies, softmax; and the leader's products
      }
      mbar_init(c.bar(B_STAT), 4);
      mbar_init(c.bar(B_READ), 4);
      mbar_init(c.bar(B_NEXT), 1);
      mbar_init(c.bar(B_ASKED), 1);
      mbar_init(c.bar(B_FIN), 1);
      fence_mbar_init();
      prefetch_tensormap(&maps.q_nope);
      prefetch_tensormap(&maps.q_pe);
      prefetch_tensormap(&maps.k_nope);
      prefetch_tensormap(&maps.k_pe);
      prefetch_tensormap(&maps.v);
    }
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc_of<kCtas>(c.sbase + kOffTmem);
  }
  // The work before this launch is complete before anything of it is read or replaced.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (kCtas > 1) cluster_sync();  // the peer's barriers are initialised before any arrival there
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
    if (warp == 0) {
      load_items(c, a, maps, lane);
    } else if (warp == 1) {
      if (c.rank == 0) issue_products(c, a, tmem);
    } else if (warp == 3) {
      if (c.rank == 0)
        schedule(c, a, work_of<kCtas>(a, blocks), own, lane);
      else
        receive(c, lane);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax_items(c, a, (warp - 4) >> 2, tmem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (kCtas > 1) cluster_sync();  // every product is read
  tc_fence_after();
  if (kCtas > 1 && c.rank > 0 && warp == 1) c.wait_limited(B_FIN, 0);  // the leader's last arrival here
  __syncwarp();
  if (warp == 1) tmem_dealloc_of<kCtas>(tmem);
  if (kCtas > 1) cluster_sync();
}

// ------------------------------------------------------------------ parts

// lse = ln sum_k e^lse_k, out = sum_k e^(lse_k - lse) out_k over the parts of a row; a
// warp a row, so that all rows' loads are on their way at once, four parts at a time.  500
// rows of 16 heads in 4 parts over 20000 keys: 79 us, 73 without the merge.  No more than
// eight CTAs an SM, which go on to further rows (kOn) where there can be more: each looks
// its rows' request up, which takes longer than a row (130 rows each of 4 requests over 130
// keys, 16 heads, none in parts: 17.8 us with a CTA for every 8 rows that there can be, 13.9
// so, 9.1 without the launch; a long request among those of 64 rows, 32 heads, 49.1 and
// 43.5).  Without the loop where it is not needed: 300 rows of 19 heads over 20000 keys 77.2,
// with it 78.2; 16 rows of 4 heads over 2000 11.9 and 12.1.
constexpr int kMergeRows = 8;  // of a CTA at a time
constexpr int kMergeCtas = 8;  // of an SM
template <int kItemRows, bool kOn>
__global__ void __launch_bounds__(32 * kMergeRows) merge_parts_kernel(const Args a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = (int)blockIdx.x / a.tiles;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Item it;
  Walk walk;
  if (!find_block<kItemRows, false>(a, a.batch, (int)blockIdx.x - head * a.tiles, walk, lane, &it)) return;
  if (it.parts == 1) return;  // its results are there
  int row = it.row0 + (int)blockIdx.y * kMergeRows + warp;
  if (row >= it.end) return;
  do {
    const int64_t token = it.q0 + row, at = token * a.heads + head, stride = (int64_t)a.tokens_q * a.heads;
    const float mine = lane < it.parts ? __ldcg(a.part_lse + lane * stride + at) : -CUDART_INF_F;  // at most 32 parts
    const float4* x = reinterpret_cast<const float4*>(a.part_out + at * 128) + lane;
    float4 v[4];  // the first ones are on their way with the lse
    auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k0 + k < it.parts) v[k] = __ldcg(x + (k0 + k) * stride * 32);
    };
    fetch(0);
    float top = mine;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float base = top == -CUDART_INF_F ? 0.f : top;
    float w = expf(mine - base), sum = w;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    w = sum == 0.f ? 0.f : w / sum;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < it.parts; k0 += 4) {
      if (k0 > 0) fetch(k0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
        const float l = __shfl_sync(0xffffffffu, mine, (k0 + k) & 31);
        if (l == -CUDART_INF_F) continue;  // it has not been written
        o.x += f * v[k].x;
        o.y += f * v[k].y;
        o.z += f * v[k].z;
        o.w += f * v[k].w;
      }
    }
    uint16_t* out = a.out + token * a.out_ts + head * a.out_hs + 4 * lane;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack(o.x, o.y), pack(o.z, o.w));
    if (lane == 0) a.lse[at] = sum == 0.f ? -CUDART_INF_F : base + logf(sum);
    row += (int)gridDim.y * kMergeRows;
  } while (kOn && row < it.end);
}

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

// bf16 [tokens, heads, cols] read in boxes of `box_rows` tokens x 64 columns of one head
static bool make_map(CUtensorMap* map, const HeadRows& x, int64_t cols, int64_t heads, int64_t tokens, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)x.head_stride * 2, (cuuint64_t)x.token_stride * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x.p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row blocks: at most this many exist
static int items_of_a_head(int num_tokens_q, int batch, int item_rows) {
  const int owners = std::min(batch, num_tokens_q);  // requests with a row, at most
  return (num_tokens_q - owners) / item_rows + owners;
}

constexpr int kMostParts = 32;
constexpr int64_t kPartRowBytes = (128 + 1) * 4, kPartBytes = 64 << 20;

// Parts of a row block's keys, at most: enough to give every CTA an item, of 256 keys or
// more.  In us, not cut, of 1024, 512 and 256 keys at least: a row over 2000 keys, 16 heads,
// 26.6, 26.6, 17.8, 16.9 (16.0 since the merge starts earlier); over 16000 165, 36, 36, 36; 16
// rows over 2000 keys, 4 heads, 26.4, 26.4, 16.7, 14.1 (13.5); 300 rows over 20000 keys, 19
// heads, 228, 79, 79, 78.
// The keys may be one request's: where few requests give few items they are cut as their
// lengths ask for (on the device), within 64 MB of results, from kUnevenKeys on.  Even
// requests pay 5 us for a merge of nothing; one that has nearly all of 1000 keys gains 2
// (8 of a row, 16 heads, 17.8 to 15.5), of 1700 5 (4 of 64 rows, 21.0 to 15.9), of 4200 13.
constexpr int kUnevenKeys = 6 * kPartKeys;
template <int kCtas>
static int parts_of(int num_tokens_q, int num_tokens_k, int batch, int num_heads, int sms) {
  const int64_t items = std::max<int64_t>(1, (int64_t)items_of_a_head(num_tokens_q, batch, Form<kCtas>::kItemRows) * num_heads);
  int64_t parts = std::min<int64_t>(sms / kCtas / items, num_tokens_k / batch / kPartKeys);
  if (batch > 1 && batch <= 32 && items <= 2 * sms / kCtas && num_tokens_k >= kUnevenKeys) {
    const int64_t bytes = (int64_t)std::max(1, num_tokens_q) * num_heads * kPartRowBytes;
    parts = std::max(parts, std::min<int64_t>(num_tokens_k / kPartKeys, kPartBytes / bytes));
  }
  return (int)std::max<int64_t>(1, std::min<int64_t>(parts, kMostParts));
}
// Pairs of CTAs, or one CTA an item: by the rows and keys of a request, on average.
// Measured in us (128 heads; one CTA, pair): 8 requests of 512 rows 131 and 138, 16 of 300
// rows 178 and 208, one of 1024 rows 57 and 57, of 1537 116 and 111, of 2048 163 and 137; with
// a prefix, 8 of 200 rows and 1000 keys 150 and 145, one of 512 and 2800 112 and 85; 16 of
// 64 rows and 1000 keys 200 and 262 (half of a pair has no row of 128 or fewer).  The host
// knows the totals alone, so a prompt among empty or short requests is taken for short ones:
// 8192 rows alone 1600, padded to 64 requests 2190; 4 of 2048 531, padded to 64 628.
static bool in_pairs(int num_tokens_q, int num_tokens_k, int batch) {
  return num_tokens_q / batch > kRows && num_tokens_k / batch > 600;
}

// Keys and values of a group of heads (a request's, on average).  16 and 128 heads of one
// prompt of 8192: 24 MB 229 and 1494 us, 32 MB 193 and 1460, 48 MB 194 and 1578; one head
// after the other 237 and 1598.
constexpr int64_t kGroupBytes = 32 << 20;
static int group_of(int num_tokens_k, int batch, int num_heads) {
  const int64_t bytes = 512 * ((int64_t)std::max(1, num_tokens_k) / batch) * num_heads;
  const int64_t groups = std::max<int64_t>(1, (bytes + kGroupBytes - 1) / kGroupBytes);
  return (int)((num_heads + groups - 1) / groups);
}

// Clusters: one for each item that there can be, but no more than twice those of rows that
// are all one request's, or eight an SM.  With more items than clusters each takes several.
// (A batch padded with empty requests would else start many for nothing: 2048 rows of 4
// requests among 512, 128 heads, took 2166 us, now 82; as a batch of 4, in the same form, they
// take 71.  Two an SM left 4 requests of 64 rows over 1000 to 4000 keys at 149 us, eight 138.)
template <int kCtas>
static int64_t clusters_of(const PrefillCall& p, const Args& a, int sms) {
  const int64_t full = ((int64_t)p.num_tokens_q + Form<kCtas>::kItemRows - 1) / Form<kCtas>::kItemRows * a.heads * a.parts;
  return std::min<int64_t>((int64_t)a.tiles * a.heads * a.parts, std::max<int64_t>(2 * full, 8 * sms / kCtas));
}

template <int kCtas>
static cudaError_t launch(const PrefillCall& p, Args a, Device dev, cudaStream_t stream) {
  using F = Form<kCtas>;
  constexpr auto kernel = prefill_kernel<kCtas>;
  static OncePerDevice once;
  const cudaError_t e =
      once.run(dev.id, [] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
  if (e != cudaSuccess) return e;
  Maps m;
  // without a key no box of the keys is ever loaded: any valid map will do
  const bool keys = p.num_tokens_k > 0;
  const int64_t tk = keys ? p.num_tokens_k : 1;
  if (!make_map(&m.q_nope, p.q_nope, 128, p.num_heads, p.num_tokens_q, kRows) ||
      !make_map(&m.q_pe, p.q_pe, 64, p.num_heads, p.num_tokens_q, kRows) ||
      !make_map(&m.k_nope, keys ? p.k_nope : p.q_nope, 128, p.num_heads, tk, 64) ||
      !make_map(&m.k_pe, keys ? p.k_pe : p.q_pe, 64, 1, tk, 64) ||
      !make_map(&m.v, keys ? p.v : p.q_nope, 128, p.num_heads, tk, F::kKeys))
    return cudaErrorNotSupported;
  a.tiles = items_of_a_head(p.num_tokens_q, p.batch, F::kItemRows);
  a.slots = dev.sms / kCtas;
  a.parts = parts_of<kCtas>(p.num_tokens_q, p.num_tokens_k, p.batch, p.num_heads, dev.sms);
  a.group = group_of(p.num_tokens_k, p.batch, p.num_heads);
  a.part_out = static_cast<float*>(p.workspace);
  a.part_lse = a.part_out + (int64_t)a.parts * p.num_tokens_q * p.num_heads * 128;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters_of<kCtas>(p, a, dev.sms) * kCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t main = cudaLaunchKernelEx(&cfg, kernel, m, a);
  if (main != cudaSuccess || a.parts == 1) return main;
  const int row_blocks = a.tiles * a.heads, row_groups = (std::min(F::kItemRows, p.num_tokens_q) + kMergeRows - 1) / kMergeRows;
  const int at_once = std::min(row_groups, std::max(1, kMergeCtas * dev.sms / row_blocks));
  cfg.gridDim = dim3((unsigned)row_blocks, (unsigned)at_once);
  cfg.blockDim = dim3(32 * kMergeRows);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  if (at_once < row_groups) return cudaLaunchKernelEx(&cfg, merge_parts_kernel<F::kItemRows, true>, a);
  return cudaLaunchKernelEx(&cfg, merge_parts_kernel<F::kItemRows, false>, a);
}

}  // namespace prefill

// Arguments are checked by the caller; cudaErrorNotSupported: the tensor-map
// encoder is unavailable or rejected the operands.
cudaError_t launch_prefill(const PrefillCall& p, Device dev, cudaStream_t stream) {
  using namespace prefill;
  Args a{};
  a.cu_q = p.cu_q;
  a.cu_k = p.cu_k;
  a.v = static_cast<const uint16_t*>(p.v.p);
  a.out = static_cast<uint16_t*>(const_cast<void*>(p.out.p));
  a.lse = p.lse;
  a.v_ts = p.v.token_stride;
  a.v_hs = p.v.head_stride;
  a.out_ts = p.out.token_stride;
  a.out_hs = p.out.head_stride;
  a.batch = p.batch;
  a.heads = p.num_heads;
  a.tokens_q = p.num_tokens_q;
  a.tokens_k = p.num_tokens_k;
  a.causal = p.causal;
  a.scale_log2 = p.scale * 1.44269504088896340736f;
  return in_pairs(p.num_tokens_q, p.num_tokens_k, p.batch) ? launch<2>(p, a, dev, stream) : launch<1>(p, a, dev, stream);
}

// Launch bound: the small form's CTAs, at most
int prefill_items(int num_tokens_q, int batch) {
  return prefill::items_of_a_head(num_tokens_q, batch, prefill::Form<1>::kItemRows);
}

PrefillForm prefill_form(int num_tokens_q, int num_tokens_k, int batch, int num_heads, int sms) {
  using namespace prefill;
  const bool pairs = in_pairs(num_tokens_q, num_tokens_k, batch);
  PrefillForm f;
  f.item_rows = pairs ? Form<2>::kItemRows : Form<1>::kItemRows;
  f.parts = pairs ? parts_of<2>(num_tokens_q, num_tokens_k, batch, num_heads, sms)
                  : parts_of<1>(num_tokens_q, num_tokens_k, batch, num_heads, sms);
  f.group = group_of(num_tokens_k, batch, num_heads);
  // what the parts write; 0: the keys are not cut
  f.workspace = f.parts == 1 ? 0 : align256((size_t)f.parts * num_tokens_q * num_heads * kPartRowBytes);
  return f;
}

// Enough for every call of up to these sizes (one call's need does not grow with each of
// them): no call has more parts than kMostParts or the pieces of kPartKeys in all keys, and
// parts that are there to occupy the SMs write no more than their rows at a time, parts of
// uneven requests no more than kPartBytes.
size_t prefill_workspace(int num_tokens_q, int num_tokens_k, int batch, int num_heads, int sms) {
  using namespace prefill;
  const int64_t parts = std::min(kMostParts, num_tokens_k / kPartKeys);
  if (parts < 2) return 0;
  const int64_t busy = (int64_t)sms * Form<1>::kItemRows * kPartRowBytes;
  const int64_t most = batch > 1 ? std::max(busy, kPartBytes) : busy;
  return align256((size_t)std::min(parts * num_tokens_q * num_heads * kPartRowBytes, most));
}

cudaError_t prefill_read_error(int* code, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(code, prefill::g_prefill_error, sizeof(int));
  if (e != cudaSuccess || !reset) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(prefill::g_prefill_error, &zero, sizeof(int));
}

}  // namespace mla
