// Latent attention in its expanded form, for prompts: every head has its own
// 128-wide keys and values, and the 64 rotary key columns are one row shared by
// all heads (sglang trtllm_mla_backend.py, forward_extend: ragged attention of
// head dims 192 / 128 with lse; tokenspeed trtllm_mla.py, forward_extend).
//
//   s_j = scale (q_nope . k_nope_j + q_pe . k_pe_j),   out = softmax(s) V,   lse = ln sum e^s
//
// One CTA per item: 256 query rows of one request and head, as two tiles of 128
// rows whose products and softmax alternate.  Per 128 keys and tile
//   S = Q K^T    (M = 128, N = 128, K = 192)  operands in shared memory -> TMEM
//   P = 2^(c S - m) in registers, bf16, written over S
//   O += P V     (M = 128, N = 128, K = 128)  P from TMEM, V from shared memory
// A thread of the softmax owns one query row, so its maximum and sum need no
// exchange.  While one tile's softmax runs, the tensor core has the other
// tile's products.  The running maximum only moves when a score exceeds it by
// 2^8 (P stays below 256, which bf16 and the fp32 sums hold); then that warp
// rescales its rows of O, which no product uses at that time: the products of a
// tile run in order, so S(j) in TMEM means that P V (j - 1) is done.
//
// P enters the second product in bf16 (half a step: 2^-9 of each weight, of
// random sign, below the rounding of the bf16 output); row sums and lse use the
// unrounded values.
//
// TMEM (512 columns): S / P of both tiles [0, 256), O of both tiles [256, 512).
// Shared memory: Q (2 x 48 KB) and a ring of eight 16 KB slots, each 128 keys x
// 64 columns in the 128-byte swizzle: a key tile takes three (two of k_nope, one
// of k_pe), a value tile two.
//
// Masked places.  Scores past a row's last key are replaced by -inf, so keys
// there may hold anything.  Values there are multiplied by P = 0, which leaves
// NaN of an infinity or a NaN; so two warps look through the value tiles that
// some row does not see whole, and put zeros in the place of what is not finite.
// The rows that do see such a value get it in the epilogue.
//
// Warps: 0 TMA, 1 MMA, 2-3 value scan, 4-7 softmax of the first tile, 8-11 of
// the second.  Waits are bounded: on timeout the error word is set, every role
// stops, copies and products in flight are awaited, TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <mutex>

#include "../../include/mla_decode.h"
#include "mla_internal.h"
#include "per_device.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace prefill {

using namespace mla::ptx;

__device__ int g_prefill_error;

constexpr int kRows = 128;             // query rows of a tile
constexpr int kItemRows = 2 * kRows;   // ... and of an item
constexpr int kKeys = 128;             // keys of a step
constexpr int kSlot = kKeys * 128;     // bytes of a ring slot, and of a Q box
constexpr int kSlots = 8;
constexpr int kKSlots = 3, kVSlots = 2, kStepSlots = kKSlots + kVSlots;
constexpr int kQTile = 3 * kSlot;
constexpr int kOffQ = 0;
constexpr int kOffRing = 2 * kQTile;
constexpr int kOffBars = kOffRing + kSlots * kSlot;
constexpr int kThreads = 384;
constexpr int kRegsLoad = 56, kRegsSoftmax = 224;  // 128 x 56 + 256 x 224 = 384 x 168, the launch's registers
constexpr float kRescaleLog2 = 8.0f;
constexpr long long kTimeoutCycles = 2000000000LL;

enum Bar : int {
  B_Q = 0,                    // [tile]
  B_FULL = B_Q + 2,           // [slot]
  B_EMPTY = B_FULL + kSlots,  // [slot]
  B_S = B_EMPTY + kSlots,     // [tile] scores are in TMEM
  B_P = B_S + 2,              // [tile] weights are in TMEM, O is rescaled
  B_O = B_P + 2,              // [tile] the tile's products are done
  B_RAW = B_O + 2,            // [2 w + step parity] half w of a value tile landed, for the scan
  B_FIN = B_RAW + 4,          // every product is done
  B_COUNT
};
constexpr int kOffTmem = kOffBars + B_COUNT * 8;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kOffPoison = kOffAbort + 4;
constexpr int kOffItem = (kOffPoison + 4 + 15) / 16 * 16;
constexpr int kSmem = kOffItem + 32 + 1024;  // + alignment slack
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
  int32_t tiles;   // items of a head: at most this many exist
  int32_t causal;
  float scale_log2;  // scale * log2(e)
};

struct Item {
  int q0, lq, k0, lk;  // the request's rows and keys
  int head, row0;      // first query row of the item within the request
};

// What one tile (of 128 rows) of an item computes.
struct Tile {
  int row0, rows;  // within the request
  int steps;       // key tiles with a visible key
  int masked;      // first of them that some row does not see whole
};

__device__ __forceinline__ int visible(const Item& it, int causal, int row) {
  return causal ? max(0, min(it.lk, it.lk - it.lq + 1 + row)) : it.lk;
}
__device__ __forceinline__ Tile tile_of(const Item& it, int causal, int t) {
  Tile d;
  d.row0 = it.row0 + t * kRows;
  d.rows = min(kRows, it.lq - d.row0);
  d.steps = d.masked = 0;
  if (d.rows <= 0) {
    d.rows = 0;
  } else {
    d.steps = (visible(it, causal, d.row0 + d.rows - 1) + kKeys - 1) / kKeys;
    d.masked = visible(it, causal, d.row0) / kKeys;
  }
  return d;
}

// Item `idx` of a head: requests own ceil(rows / 256) items each, those with the
// most keys first.  Found by a warp over the offsets; false: there is no such item.
// A request whose offsets break the rules, by themselves or by beginning before an
// earlier one's end, owns none.
__device__ bool find_item(const Args& a, int idx, int lane, Item* it) {
  int items = 0, end = 0;  // of the requests so far
  bool bad_q = false, bad_k = false, found = false;
  for (int base = 0; base < a.batch; base += 32) {
    const int b = base + lane;
    int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    if (b < a.batch) {
      q0 = __ldg(a.cu_q + b);
      q1 = __ldg(a.cu_q + b + 1);
      k0 = __ldg(a.cu_k + b);
      k1 = __ldg(a.cu_k + b + 1);
    }
    int before = q1;  // the latest end of the requests before this one
#pragma unroll
    for (int d = 1; d < 32; d *= 2) before = max(before, __shfl_up_sync(0xffffffffu, before, d) * (lane >= d));
    const int last = max(end, __shfl_sync(0xffffffffu, before, 31));
    before = __shfl_up_sync(0xffffffffu, before, 1);
    before = max(end, lane ? before : 0);
    end = last;
    const bool ok_q = q0 >= before && q0 <= q1 && q1 <= a.tokens_q, ok_k = k0 >= 0 && k0 <= k1 && k1 <= a.tokens_k;
    if (b < a.batch) {
      bad_q |= !ok_q;
      bad_k |= !ok_k;
    }
    int upto = ok_q && ok_k ? (q1 - q0 + kItemRows - 1) / kItemRows : 0;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) upto += __shfl_up_sync(0xffffffffu, upto, d) * (lane >= d);
    upto += items;
    const unsigned hit = __ballot_sync(0xffffffffu, upto > idx);
    if (hit && !found) {
      found = true;
      const int src = __ffs(hit) - 1;
      it->q0 = __shfl_sync(0xffffffffu, q0, src);
      it->lq = __shfl_sync(0xffffffffu, q1, src) - it->q0;
      it->k0 = __shfl_sync(0xffffffffu, k0, src);
      it->lk = __shfl_sync(0xffffffffu, k1, src) - it->k0;
      it->row0 = (__shfl_sync(0xffffffffu, upto, src) - 1 - idx) * kItemRows;
    }
    items = __shfl_sync(0xffffffffu, upto, 31);
    if (found && idx != 0) break;  // the first item's finder looks at every request
  }
  if (idx == 0 && (bad_q || bad_k)) atomicCAS(&g_prefill_error, 0, bad_q ? 0xA01 : 0xA02);
  return found;
}

__device__ __forceinline__ uint32_t flag_load(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void flag_store(uint32_t addr, uint32_t v) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

struct Ctx {
  uint32_t sbase;
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

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

struct Maps {
  CUtensorMap q_nope, q_pe, k_nope, k_pe, v;
};

// ------------------------------------------------------------------ TMA

// The value tiles from step scan_from on complete on barriers of the scan, which
// then fills the slot's own: the products wait for one barrier a slot, and no one
// waits for a phase that another may leave behind.
__device__ __forceinline__ int raw_bar(int half, int scans) { return B_RAW + 2 * half + (scans & 1); }

__device__ void load_item(const Ctx& c, const Maps& m, const Item& it, const Tile& ta, const Tile& tb, int scan_from) {
  const int steps = max(ta.steps, tb.steps);
  int slot = 0, issued = 0;
  uint32_t phase = 0;
  bool ok = true;
  auto load_q = [&](int t, const Tile& d) {
    if (d.steps == 0) return;
    const uint32_t dst = c.sbase + kOffQ + t * kQTile, bar = c.bar(B_Q + t);
    const int row = it.q0 + d.row0;
    mbar_arrive_expect_tx(bar, kQTile);
    tma_3d(dst, &m.q_nope, bar, 0, it.head, row);
    tma_3d(dst + kSlot, &m.q_nope, bar, 64, it.head, row);
    tma_3d(dst + 2 * kSlot, &m.q_pe, bar, 0, it.head, row);
  };
  load_q(0, ta);
  for (int j = 0; ok && j < steps; ++j) {
    const int row = it.k0 + j * kKeys;
    for (int i = 0; ok && i < kStepSlots; ++i) {
      if (!(ok = c.wait(B_EMPTY + slot, phase ^ 1, 0xA11))) break;
      const bool scan = i >= kKSlots && j >= scan_from;
      const uint32_t dst = c.sbase + kOffRing + slot * kSlot;
      const uint32_t bar = c.bar(scan ? raw_bar(i - kKSlots, j - scan_from) : B_FULL + slot);
      mbar_arrive_expect_tx(bar, kSlot);
      if (i < 2)
        tma_3d(dst, &m.k_nope, bar, 64 * i, it.head, row);
      else if (i == 2)
        tma_3d(dst, &m.k_pe, bar, 0, 0, row);
      else
        tma_3d(dst, &m.v, bar, 64 * (i - 3), it.head, row);
      ++issued;
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1;
      }
      if (j == 0 && i == 2) load_q(1, tb);
    }
  }
  // every copy has landed before this CTA may leave
  if (!ok) {
    if (ta.steps) c.wait_limited(B_Q, 0);
    if (tb.steps) c.wait_limited(B_Q + 1, 0);
    for (int i = max(0, issued - kSlots); i < issued; ++i) {
      const int scans = i / kStepSlots - scan_from, half = i % kStepSlots - kKSlots;
      if (scans >= 0 && half >= 0)
        c.wait_limited(raw_bar(half, scans), (scans >> 1) & 1);
      else
        c.wait_limited(B_FULL + i % kSlots, (i / kSlots) & 1);
    }
  }
}

// ------------------------------------------------------------------ MMA

// Operand descriptors differ in the start address alone (the low word).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (kSwizzle128B << 29);
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lbo) {
  const uint32_t low = ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
  return static_cast<uint64_t>(kDescHigh) << 32 | low;
}

__device__ void issue_products(const Ctx& c, uint32_t tmem, const Tile& ta, const Tile& tb) {
  constexpr uint32_t kIdescS = idesc_f32acc(kRows, kKeys, 0, 0, 1), kIdescO = idesc_f32acc(kRows, 128, 0, 1, 1);
  const int steps[2] = {ta.steps, tb.steps};
  const int total = max(ta.steps, tb.steps);
  bool ok = true, q_here[2] = {false, false};
  for (int j = 0; ok && j <= total; ++j) {
    bool k_here = false, v_here = false;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (!ok) break;
      if (j > 0 && j - 1 < steps[t]) {
        // ---- O += P V of step j - 1
        const int first = (j - 1) * kStepSlots + kKSlots;
        if (!v_here) {
          for (int i = first; ok && i < first + kVSlots; ++i) ok = c.wait(B_FULL + i % kSlots, (i / kSlots) & 1, 0xA12);
          v_here = true;
        }
        if (!ok || !(ok = c.wait(B_P + t, (j - 1) & 1, 0xA14))) break;
        tc_fence_after();
        // the value tile's two slots are neighbours in the ring's numbering, not always in memory
        const uint32_t v0 = c.sbase + kOffRing + (first % kSlots) * kSlot;
        const uint32_t v1 = c.sbase + kOffRing + ((first + 1) % kSlots) * kSlot;
        constexpr uint32_t kIdescHalf = idesc_f32acc(kRows, 64, 0, 1, 1);
        if (v1 == v0 + kSlot) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts(tmem + TM_O + 128 * t, tmem + TM_S + 128 * t + 8 * kk, desc(v0 + kk * 2048, kSlot), kIdescO,
                   j > 1 || kk > 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk) {
            mma_ts(tmem + TM_O + 128 * t, tmem + TM_S + 128 * t + 8 * kk, desc(v0 + kk * 2048, kSlot), kIdescHalf,
                   j > 1 || kk > 0);
            mma_ts(tmem + TM_O + 128 * t + 64, tmem + TM_S + 128 * t + 8 * kk, desc(v1 + kk * 2048, kSlot), kIdescHalf,
                   j > 1 || kk > 0);
          }
        }
        if (j == steps[t]) mma_commit(c.bar(B_O + t));
        if (t == 1 || j - 1 >= steps[1])  // its last reader
          for (int i = first; i < first + kVSlots; ++i) mma_commit(c.bar(B_EMPTY + i % kSlots));
      }
      if (j < steps[t]) {
        // ---- S = Q K^T of step j
        const int first = j * kStepSlots;
        if (!k_here) {
          for (int i = first; ok && i < first + kKSlots; ++i) ok = c.wait(B_FULL + i % kSlots, (i / kSlots) & 1, 0xA15);
          k_here = true;
        }
        if (ok && !q_here[t]) {
          ok = c.wait(B_Q + t, 0, 0xA16);
          q_here[t] = true;
        }
        if (!ok) break;
        tc_fence_after();
        const uint32_t qa = c.sbase + kOffQ + t * kQTile;
#pragma unroll
        for (int kk = 0; kk < 12; ++kk) {
          const uint32_t ka = c.sbase + kOffRing + ((first + kk / 4) % kSlots) * kSlot;
          mma_ss(tmem + TM_S + 128 * t, desc(qa + (kk / 4) * kSlot + (kk % 4) * 32, 16), desc(ka + (kk % 4) * 32, 16),
                 kIdescS, kk > 0);
        }
        mma_commit(c.bar(B_S + t));
        if (t == 1 || j >= steps[1])
          for (int i = first; i < first + kKSlots; ++i) mma_commit(c.bar(B_EMPTY + i % kSlots));
      }
    }
  }
  // every product is done before TMEM is released
  mma_commit(c.bar(B_FIN));
  c.wait_limited(B_FIN, 0);
}

// ------------------------------------------------------------------ value scan

// Zeros in the place of what is not finite, in the value tiles from step
// scan_from on; warp w looks after the tile's columns 64 w .. 64 w + 63.
__device__ void scan_values(const Ctx& c, const Item& it, int steps, int scan_from, int w, int lane) {
  for (int j = scan_from; j < steps; ++j) {
    const int slot = (j * kStepSlots + kKSlots + w) % kSlots, scans = j - scan_from;
    if (!c.wait_warp(raw_bar(w, scans), (scans >> 1) & 1, 0xA13)) return;
    const uint32_t base = c.sbase + kOffRing + slot * kSlot + lane * 16;
    bool seen = false;
#pragma unroll 4
    for (int i = 0; i < kSlot / 512; ++i) {
      uint4 x = ld_shared_v4(base + i * 512);
      constexpr uint32_t kExp = 0x7F807F80u;
      const uint32_t b0 = __vcmpeq2(x.x & kExp, kExp), b1 = __vcmpeq2(x.y & kExp, kExp), b2 = __vcmpeq2(x.z & kExp, kExp),
                     b3 = __vcmpeq2(x.w & kExp, kExp);
      if (b0 | b1 | b2 | b3) {
        x.x &= ~b0;
        x.y &= ~b1;
        x.z &= ~b2;
        x.w &= ~b3;
        st_shared_v4(base + i * 512, x);
        seen |= j * kKeys + i * 4 + (lane >> 3) < it.lk;  // a slot's row is 128 bytes
      }
    }
    if (seen) flag_store(c.sbase + kOffPoison, 1);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar(B_FULL + slot));
  }
}

// ------------------------------------------------------------------ softmax

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
#define MLA_I8(b) "r"(r[b + 0]), "r"(r[b + 1]), "r"(r[b + 2]), "r"(r[b + 3]), "r"(r[b + 4]), "r"(r[b + 5]), \
                  "r"(r[b + 6]), "r"(r[b + 7])
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&r)[16]) {
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

// Sum of what is not finite among the values of keys [from, to) in one column: they
// weigh something, so an infinity or a NaN is what a row that sees them gets.
__device__ __noinline__ float non_finite(const uint16_t* v, int64_t stride, int from, int to) {
  float sum = 0.f;
  for (int key = from; key < to; ++key) {
    const uint32_t bits = v[key * stride];
    if ((bits & 0x7F80u) == 0x7F80u) sum += __uint_as_float(bits << 16);
  }
  return sum;
}

__device__ void softmax_tile(const Ctx& c, const Args& a, const Item& it, const Tile& d, int t, int scan_from, uint32_t tmem) {
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const int row = d.row0 + quad * 32 + lane;  // within the request
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t ts = tmem + lanes + TM_S + 128 * t, to = tmem + lanes + TM_O + 128 * t;
  const int seen = visible(it, a.causal, min(row, it.lq - 1));
  const float slack = kRescaleLog2 / a.scale_log2;
  float top = -CUDART_INF_F, sum = 0.f;  // the running maximum (of S) and sum
  for (int j = 0; j < d.steps; ++j) {
    if (!c.wait_warp(B_S + t, j & 1, 0xA18)) return;
    tc_fence_after();
    uint32_t s[4][32];
#pragma unroll
    for (int q = 0; q < 4; ++q) tmem_ld32_async(ts + 32 * q, s[q]);
#pragma unroll
    for (int q = 0; q < 4; ++q) tmem_wait_ld32(s[q]);
    if (j >= d.masked) {
      const int left = seen - j * kKeys;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (32 * q + i >= left) s[q][i] = 0xFF800000u;  // -inf
    }
    float high[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      high[q] = __uint_as_float(s[q][0]);
#pragma unroll
      for (int i = 1; i < 32; ++i) high[q] = fmaxf(high[q], __uint_as_float(s[q][i]));
    }
    const float here = fmaxf(fmaxf(high[0], high[1]), fmaxf(high[2], high[3]));
    const bool move = here > top + slack;
    if (__any_sync(0xffffffffu, move)) {
      const float factor = move ? ex2_approx((top - here) * a.scale_log2) : 1.f;
      if (move) top = here;
      sum *= factor;
      if (j > 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t o[32];
          tmem_ld32(to + 32 * q, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
          tmem_st32(to + 32 * q, o);
        }
      }
    }
    const float base = top == -CUDART_INF_F ? 0.f : top * a.scale_log2;
    float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t p[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x = ex2_approx(fmaf(__uint_as_float(s[q][2 * i]), a.scale_log2, -base));
        const float y = ex2_approx(fmaf(__uint_as_float(s[q][2 * i + 1]), a.scale_log2, -base));
        add[i & 3] += x + y;
        p[i] = pack(x, y);
      }
      tmem_st16_async(ts + 16 * q, p);
    }
    sum += (add[0] + add[1]) + (add[2] + add[3]);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar(B_P + t));
  }
  // ---- epilogue
  if (d.steps > 0) {
    if (!c.wait_warp(B_O + t, 0, 0xA19)) return;
    tc_fence_after();
  }
  const bool mine = row < it.lq;
  const bool none = sum == 0.f;  // no key, or scores of -inf alone
  const float inv = 1.f / sum;
  const bool poison = flag_load(c.sbase + kOffPoison) != 0;
  const int64_t token = it.q0 + row;
  uint16_t* out = a.out + token * a.out_ts + it.head * a.out_hs;
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    uint32_t r[32];
    if (d.steps > 0) tmem_ld32(to + 32 * q, r);
    float o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : __uint_as_float(r[i]) * inv;
    if (poison && mine && !none) {
      const uint16_t* v = a.v + it.k0 * a.v_ts + it.head * a.v_hs + 32 * q;
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] += non_finite(v + i, a.v_ts, scan_from * kKeys, seen);
    }
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = pack(o[2 * i], o[2 * i + 1]);
    if (mine) {
      store32(out + 32 * q, p, wide);
      store32(out + 32 * q + 16, p + 8, wide);
    }
  }
  if (mine) {
    const float base = top == -CUDART_INF_F ? 0.f : top * a.scale_log2;
    a.lse[token * a.heads + it.head] = none ? -CUDART_INF_F : fmaf(base, CUDART_LN2_F, logf(sum));
  }
}

__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctx c;
  c.sbase = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* slot = reinterpret_cast<volatile int*>(smem + kOffItem);  // the item; [6]: whether there is one
  if (warp == 0) {
    Item it{};
    const int idx = (int)(blockIdx.x % a.tiles);
    const bool found = find_item(a, idx, lane, &it);
    if (lane == 0) {
      slot[0] = it.q0;
      slot[1] = it.lq;
      slot[2] = it.k0;
      slot[3] = it.lk;
      slot[4] = it.row0;
      slot[6] = found;
      flag_store(c.sbase + kOffAbort, 0);
      flag_store(c.sbase + kOffPoison, 0);
      for (int t = 0; t < 2; ++t) {
        mbar_init(c.bar(B_Q + t), 1);
        mbar_init(c.bar(B_S + t), 1);
        mbar_init(c.bar(B_P + t), 4);
        mbar_init(c.bar(B_O + t), 1);
      }
      for (int i = 0; i < kSlots; ++i) {
        mbar_init(c.bar(B_FULL + i), 1);
        mbar_init(c.bar(B_EMPTY + i), 1);
      }
      for (int i = 0; i < 4; ++i) mbar_init(c.bar(B_RAW + i), 1);
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
    tmem_alloc(c.sbase + kOffTmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);
  Item it;
  it.q0 = slot[0];
  it.lq = slot[1];
  it.k0 = slot[2];
  it.lk = slot[3];
  it.row0 = slot[4];
  it.head = (int)(blockIdx.x / a.tiles);
  if (slot[6]) {
    const Tile ta = tile_of(it, a.causal, 0), tb = tile_of(it, a.causal, 1);
    // steps whose values are looked through: those that some row does not see whole
    const int scan_from = min(ta.steps ? ta.masked : INT32_MAX, tb.steps ? tb.masked : INT32_MAX);
    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
      if (warp == 0 && lane == 0) load_item(c, maps, it, ta, tb, scan_from);
      if (warp == 1 && lane == 0) issue_products(c, tmem, ta, tb);
      if (warp >= 2) scan_values(c, it, max(ta.steps, tb.steps), scan_from, warp - 2, lane);
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
      const int t = (warp - 4) >> 2;
      const Tile d = t ? tb : ta;
      if (d.rows > 0) softmax_tile(c, a, it, d, t, scan_from, tmem);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
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

// bf16 [tokens, heads, cols] read in boxes of 128 tokens x 64 columns of one head
static bool make_map(CUtensorMap* map, const HeadRows& x, int64_t cols, int64_t heads, int64_t tokens) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)x.head_stride * 2, (cuuint64_t)x.token_stride * 2};
  cuuint32_t box[3] = {64, 1, kRows};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x.p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace prefill

// Arguments are checked by the caller; cudaErrorNotSupported: the tensor-map
// encoder is unavailable or rejected the operands.
cudaError_t launch_prefill(const PrefillCall& p, Device dev, cudaStream_t stream) {
  using namespace prefill;
  static OncePerDevice once;
  const cudaError_t e = once.run(
      dev.id, [] { return cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
  if (e != cudaSuccess) return e;
  Maps m;
  // without a key no box of the keys is ever loaded: any valid map will do
  const bool keys = p.num_tokens_k > 0;
  const HeadRows k_pe{p.k_pe.p, p.k_pe.token_stride, p.k_pe.token_stride};
  if (!make_map(&m.q_nope, p.q_nope, 128, p.num_heads, p.num_tokens_q) ||
      !make_map(&m.q_pe, p.q_pe, 64, p.num_heads, p.num_tokens_q) ||
      !make_map(&m.k_nope, keys ? p.k_nope : p.q_nope, 128, p.num_heads, keys ? p.num_tokens_k : 1) ||
      !make_map(&m.k_pe, keys ? k_pe : p.q_pe, 64, 1, keys ? p.num_tokens_k : 1) ||
      !make_map(&m.v, keys ? p.v : p.q_nope, 128, p.num_heads, keys ? p.num_tokens_k : 1))
    return cudaErrorNotSupported;
  Args a;
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
  a.tiles = prefill_items(p.num_tokens_q, p.batch);
  a.causal = p.causal;
  a.scale_log2 = p.scale * 1.44269504088896340736f;
  prefill_kernel<<<(unsigned)(a.tiles * a.heads), kThreads, kSmem, stream>>>(m, a);
  return cudaGetLastError();
}

// Items of a head: one for each 256 rows of a request, at most
int prefill_items(int num_tokens_q, int batch) {
  return num_tokens_q / prefill::kItemRows + (batch < num_tokens_q ? batch : num_tokens_q);
}

// Nothing is split over the keys: no workspace.
size_t prefill_workspace(int, int, int, int, Device) { return 0; }

cudaError_t prefill_read_error(int* code, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(code, prefill::g_prefill_error, sizeof(int));
  if (e != cudaSuccess || !reset) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(prefill::g_prefill_error, &zero, sizeof(int));
}

}  // namespace mla
