// The row operators around a prompt's attention: the table of rotary positions,
// the rotation, the gather of cached latent rows, and the merge of two partial
// attention results.  Each is bound by the bytes it moves; each is launched as a
// programmatic dependent of the work before it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/mla_decode.h"
#include "mla_internal.h"
#include "mla_prompt.h"

namespace mla_pr {

__device__ int g_rows_error;

__device__ __forceinline__ void record(int code) { atomicCAS(&g_rows_error, 0, code); }

// Wait for the work before this launch, then let the next launch begin.
__device__ __forceinline__ void grid_dependency() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t to_bf16(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

constexpr int kThreads = 256;

// ------------------------------------------------------------------ table

// cos and sin of position * frequency.  A position's angle is a whole number times
// a fixed fraction of a turn, and whole turns do not matter: the fraction is held
// in 64 bits and the product taken modulo 2^64, so the reduction costs two integer
// products and is good to 2^-31 of a turn, however far (double precision, at this
// GPU's rate, would be what bounds the kernel).  The nearest quarter turn goes, and the
// rest, at most pi / 4, through the Taylor polynomials of degree 9 and 10 (their next
// terms are below 2e-9 there); the sum is off by about one unit of 2^-24.
// 163840 positions of 64 columns: 42 MB.
struct TableArgs {
  float* table;
  int64_t first, positions;
  int32_t half;        // pairs of a row
  int32_t block_rows;  // rows of a block at a time
  float magnitude;
  uint64_t turns[MLA_ROPE_MAX_DIM / 2];  // of a position, in 2^-64 of a turn
};

__device__ __forceinline__ void cos_sin(uint32_t turn, float magnitude, float* c, float* s) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float y = static_cast<float>(static_cast<int32_t>(turn - (quarter << 30))) * (2.f * CUDART_PI_F * 0x1p-32f);
  const float z = y * y;
  const float sy = fmaf(y * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), y);
  const float cy =
      fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const float c0 = quarter & 1 ? sy : cy, s0 = quarter & 1 ? cy : sy;
  *c = __uint_as_float(__float_as_uint(c0) ^ (((quarter + 1) & 2) << 30)) * magnitude;
  *s = __uint_as_float(__float_as_uint(s0) ^ ((quarter & 2) << 30)) * magnitude;
}

// kWide: four pairs a thread and row (half % 4 == 0, 16-byte rows); else one.  kRows: rows
// of a thread, four where that fills the GPU (163840 positions: 1 row 12.5 us, 4 rows 7.3;
// 4096, in a graph: 1.5 and 1.9).
template <bool kWide, int kRows>
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ TableArgs a) {
  grid_dependency();
  constexpr int kPairs = kWide ? 4 : 1;
  const int per_row = a.half / kPairs, sub = threadIdx.x / per_row, i = (threadIdx.x - sub * per_row) * kPairs;
  if (sub >= a.block_rows) return;
  uint32_t high[kPairs], low[kPairs];
#pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    high[k] = static_cast<uint32_t>(a.turns[i + k] >> 32);
    low[k] = static_cast<uint32_t>(a.turns[i + k]);
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t p = ((int64_t)blockIdx.x * kRows + r) * a.block_rows + sub;
    if (p >= a.positions) return;
    const uint32_t position = static_cast<uint32_t>(a.first + p);
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) cos_sin(position * high[k] + __umulhi(position, low[k]), a.magnitude, c + k, s + k);
    float* row = a.table + p * 2 * a.half + i;
    if (kWide) {
      *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1 % kPairs], c[2 % kPairs], c[3 % kPairs]);
      *reinterpret_cast<float4*>(row + a.half) = make_float4(s[0], s[1 % kPairs], s[2 % kPairs], s[3 % kPairs]);
    } else {
      row[0] = c[0];
      row[a.half] = s[0];
    }
  }
}

// ------------------------------------------------------------------ rotation

struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  int64_t q_ts, q_hs, qo_ts, qo_hs, k_ts, ko_ts;
  const int64_t* positions;
  const float* table;
  int64_t max_position;
  int32_t tokens, heads;  // query heads; k may be NULL
  int32_t half;
  int32_t chunks;         // of a row: threads that share it
  int32_t lanes;          // heads of a token at a time
  int32_t block_tokens;   // tokens of a block
};

constexpr int kRopeRows = 4;       // that a thread has in flight
constexpr int kRopeThreads = 128;  // 8192 tokens of 128 heads: 41.3 us (99% of a measured copy), of 256 43.3, of 512 62

// Four pairs of a row.
template <bool kNeox>
__device__ __forceinline__ uint4 load_pairs(const uint16_t* row, int chunk, int half) {
  if (!kNeox) return *reinterpret_cast<const uint4*>(row + 8 * chunk);
  const uint2 lo = *reinterpret_cast<const uint2*>(row + 4 * chunk), hi = *reinterpret_cast<const uint2*>(row + half + 4 * chunk);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
// ... rotated.
template <bool kNeox>
__device__ __forceinline__ void rotate_pairs(uint4 v, float4 c, float4 s, uint16_t* row, int chunk, int half) {
  float x[4], y[4], p[4], q[4];
  if (kNeox) {
    x[0] = bf_lo(v.x); x[1] = bf_hi(v.x); x[2] = bf_lo(v.y); x[3] = bf_hi(v.y);
    y[0] = bf_lo(v.z); y[1] = bf_hi(v.z); y[2] = bf_lo(v.w); y[3] = bf_hi(v.w);
  } else {
    x[0] = bf_lo(v.x); y[0] = bf_hi(v.x); x[1] = bf_lo(v.y); y[1] = bf_hi(v.y);
    x[2] = bf_lo(v.z); y[2] = bf_hi(v.z); x[3] = bf_lo(v.w); y[3] = bf_hi(v.w);
  }
  const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = __fsub_rn(__fmul_rn(x[i], cs[i]), __fmul_rn(y[i], sn[i]));
    q[i] = __fadd_rn(__fmul_rn(y[i], cs[i]), __fmul_rn(x[i], sn[i]));
  }
  if (kNeox) {
    *reinterpret_cast<uint2*>(row + 4 * chunk) = make_uint2(bf16x2(p[0], p[1]), bf16x2(p[2], p[3]));
    *reinterpret_cast<uint2*>(row + half + 4 * chunk) = make_uint2(bf16x2(q[0], q[1]), bf16x2(q[2], q[3]));
  } else {
    *reinterpret_cast<uint4*>(row + 8 * chunk) =
        make_uint4(bf16x2(p[0], q[0]), bf16x2(p[1], q[1]), bf16x2(p[2], q[2]), bf16x2(p[3], q[3]));
  }
}

// A thread keeps the cosines and sines of its pairs (four, or one where rows are
// not made of 16-byte pieces) and rotates them in several heads of its token; the
// first rows are on their way while the position and its cosines are found.  Each
// product and sum is rounded to fp32 on its own, as in the cache write's rotation.
template <bool kWide, bool kNeox>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  grid_dependency();
  const int chunk = threadIdx.x % a.chunks, slot = threadIdx.x / a.chunks;
  const int sub = slot / a.lanes, lane = slot - sub * a.lanes;
  const int64_t t = (int64_t)blockIdx.x * a.block_tokens + sub;
  if (sub >= a.block_tokens || t >= a.tokens) return;
  const bool key = a.k != nullptr && lane == a.lanes - 1;  // the last lane has the key as well
  const int64_t step = a.lanes * a.q_hs, out_step = a.lanes * a.qo_hs;
  const uint16_t* src = a.q + t * a.q_ts + lane * a.q_hs;
  const uint16_t* key_src = a.k + t * a.k_ts;
  uint4 v[kRopeRows], kv = make_uint4(0, 0, 0, 0);
  auto fetch = [&](int h) {
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i)
      if (h + i * a.lanes < a.heads) v[i] = load_pairs<kNeox>(src + i * step, chunk, a.half);
  };
  if (kWide) {
    fetch(lane);
    if (key) kv = load_pairs<kNeox>(key_src, chunk, a.half);
  }
  const int64_t pos = a.positions[t];
  if (pos < 0 || pos >= a.max_position) {
    if (chunk == 0 && lane == 0) record(0x801);
    return;  // nothing of this token is written
  }
  const float* row = a.table + pos * 2 * a.half;
  uint16_t* dst = a.q_out + t * a.qo_ts + lane * a.qo_hs;
  uint16_t* key_dst = a.k_out + t * a.ko_ts;
  if (kWide) {
    const float4 c = *reinterpret_cast<const float4*>(row + 4 * chunk);
    const float4 s = *reinterpret_cast<const float4*>(row + a.half + 4 * chunk);
    if (key) rotate_pairs<kNeox>(kv, c, s, key_dst, chunk, a.half);
    for (int h = lane; h < a.heads; h += kRopeRows * a.lanes) {
      if (h > lane) fetch(h);
#pragma unroll
      for (int i = 0; i < kRopeRows; ++i)
        if (h + i * a.lanes < a.heads) rotate_pairs<kNeox>(v[i], c, s, dst + i * out_step, chunk, a.half);
      src += kRopeRows * step;
      dst += kRopeRows * out_step;
    }
  } else {
    const float c = row[chunk], s = row[a.half + chunk];
    const int at0 = kNeox ? chunk : 2 * chunk, at1 = kNeox ? a.half + chunk : 2 * chunk + 1;
    auto one = [&](const uint16_t* x, uint16_t* o) {
      const float u = bf(x[at0]), v = bf(x[at1]);
      o[at0] = to_bf16(__fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s)));
      o[at1] = to_bf16(__fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s)));
    };
    if (key) one(key_src, key_dst);
    for (int h = lane; h < a.heads; h += a.lanes, src += step, dst += out_step) one(src, dst);
  }
}

// ------------------------------------------------------------------ gather

struct GatherArgs {
  const uint8_t* kv;
  const int32_t* block_table;
  const int32_t* starts;  // or nullptr: 0
  const int32_t* cu;
  uint8_t* latent;
  float* scales;
  uint16_t* k_pe;
  int64_t num_pages, bt_stride, latent_stride, scale_stride, k_pe_stride;  // outputs' strides in elements
  int32_t page_shift, batch, tokens;
  float k_scale;
};

// A warp copies four rows: it looks them up at once, a lane each (a chain: offsets, block
// table, row), then has all of them on their way, and their rotary parts and scales in
// one access for the four.  Offsets, starts and block table are read by plain loads: the
// kernel before may write them while this one is resident.  65536 rows of e4m3: 4 rows a
// warp 15.9 us, 2 rows 16.8, 8 and 16 rows four at a time 18.5 and 19.4 (fewer warps, the
// chain shows), before the accesses were joined.  Now, in a graph, by blocks of 128 and 256
// threads: 65536 rows over more data than L2 holds, bf16 25.9 us and 26.8, bf16 to codes 22.5
// and 23.3, codes 15.6 and 15.7 (77 to 88% of a measured copy's rate; e4m3 to bf16 21.6);
// 300 rows 2.5 and 3.1.
constexpr int kGatherRows = 4, kGatherThreads = 128;
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// four e4m3 codes -> four bf16 of their values times the scale
__device__ __forceinline__ uint2 widen(uint32_t v, float scale) {
  const uint32_t a = e4m3x2_f16x2(v), b = e4m3x2_f16x2(v >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return make_uint2(bf16x2(x.x * scale, x.y * scale), bf16x2(y.x * scale, y.y * scale));
}

// The request that owns row r: the last one with cu[b] <= r.  The warp narrows the
// range [0, batch] 32-fold a step.
__device__ __forceinline__ int owner(const GatherArgs& a, int r, int lane) {
  int lo = 0, n = a.batch + 1;  // cu[lo] <= r is not known for lo == 0 alone
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool le = lane * step < n && a.cu[at] <= r;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    const int end = min(lo + n, lo + (last + 1) * step);
    lo += last * step;
    n = end - lo;
  }
  return lo;
}

// 16 codes into 16 bf16 of their values times the scale
__device__ __forceinline__ void store_widened(uint4* out, uint4 v, float scale) {
  const uint2 p0 = widen(v.x, scale), p1 = widen(v.y, scale), p2 = widen(v.z, scale), p3 = widen(v.w, scale);
  out[0] = make_uint4(p0.x, p0.y, p1.x, p1.y);
  out[1] = make_uint4(p2.x, p2.y, p3.x, p3.y);
}
// A lane's 16 columns of a row through the quantiser (8 lanes share a block of 128).
__device__ __forceinline__ uint4 quantize16(const uint4 (&x)[2], float* scale) {
  float v[16];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[8 * k + 2 * e] = bf_lo(u[e]);
      v[8 * k + 2 * e + 1] = bf_hi(u[e]);
    }
  }
  uint32_t top = 0;  // magnitudes order as integers, NaN above all
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < 8; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float amax = __uint_as_float(top);
  *scale = __fdiv_rn(amax < 1e-10f ? 1e-10f : amax, 448.f);
  const float inv = __frcp_rn(*scale);
  uint32_t code[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    code[e] = e4m3x2(__fmul_rn(v[4 * e], inv), __fmul_rn(v[4 * e + 1], inv)) |
              (uint32_t)e4m3x2(__fmul_rn(v[4 * e + 2], inv), __fmul_rn(v[4 * e + 3], inv)) << 16;
  return make_uint4(code[0], code[1], code[2], code[3]);
}

template <bool kCacheE4m3, bool kOutE4m3>
__global__ void __launch_bounds__(kGatherThreads) cache_gather_kernel(const GatherArgs a) {
  constexpr int kRowBytes = kCacheE4m3 ? 576 : 1152;
  grid_dependency();
  const int lane = threadIdx.x & 31;
  const int64_t row0 = ((int64_t)blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5)) * kGatherRows;
  if (blockIdx.x == 0 && threadIdx.x < 32) {  // the offsets' rules, looked at once
    bool bad = false;
    for (int b = lane; b <= a.batch; b += 32) {
      const int c = a.cu[b];
      bad |= c < 0 || c > a.tokens || (b > 0 && c < a.cu[b - 1]);
    }
    if (bad) record(0x903);
  }
  if (row0 >= a.tokens) return;
  const uint8_t* mine = nullptr;  // lane i: where row row0 + i comes from
  {
    const int row = (int)row0 + min(lane, kGatherRows - 1);
    int b = owner(a, (int)row0, lane);
    if (b < a.batch && a.cu[b + 1] < row0 + kGatherRows) {  // the rows are not all of one request
#pragma unroll 1
      for (int i = 1; i < kGatherRows; ++i) {
        const int other = owner(a, (int)row0 + i, lane);
        if (lane >= i) b = other;
      }
    }
    if (lane < kGatherRows && row < a.tokens) {
      if (b < a.batch) {
        const int begin = a.cu[b];
        const int64_t token = (a.starts ? (int64_t)a.starts[b] : 0) + row - begin;
        if (row >= begin) {
          const int64_t block = token >> a.page_shift;
          if (token < 0 || block >= a.bt_stride) {
            record(0x901);
          } else {
            const int64_t page = a.block_table[b * a.bt_stride + block];
            if (page < 0 || page >= a.num_pages)
              record(0x902);
            else
              mine = a.kv + ((page << a.page_shift) + (token & ((1 << a.page_shift) - 1))) * kRowBytes;
          }
        }
      }
    }
  }
  // the rotary parts: a lane a 16-byte piece of row `pe_row`
  constexpr int kPieces = kCacheE4m3 ? 4 : 8;
  const int pe_row = lane / kPieces, piece = lane % kPieces;
  const auto address = reinterpret_cast<unsigned long long>(mine);
  const uint8_t* pe_src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, address, pe_row & (kGatherRows - 1)));
  const bool pe_live = pe_row < kGatherRows && pe_src;
  const uint8_t* src[kGatherRows];
  uint4 x[kGatherRows][kCacheE4m3 ? 1 : 2], pe;
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    src[i] = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, address, i));
    if (!src[i]) continue;
#pragma unroll
    for (int k = 0; k < (kCacheE4m3 ? 1 : 2); ++k)
      x[i][k] = *reinterpret_cast<const uint4*>(src[i] + ((kCacheE4m3 ? 1 : 2) * lane + k) * 16);
  }
  if (pe_live) pe = *reinterpret_cast<const uint4*>(pe_src + (kRowBytes - 16 * kPieces) + 16 * piece);

  float scales[kGatherRows];
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    if (!src[i]) continue;
    const int64_t r = row0 + i;
    if constexpr (kOutE4m3) {
      uint4* out = reinterpret_cast<uint4*>(a.latent + r * a.latent_stride) + lane;
      if constexpr (kCacheE4m3)
        *out = x[i][0];  // the codes as they are, with the cache's scale
      else
        *out = quantize16(x[i], &scales[i]);
    } else {
      uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.latent) + r * a.latent_stride) + 2 * lane;
      if constexpr (kCacheE4m3) {
        store_widened(out, x[i][0], a.k_scale);
      } else {
        out[0] = x[i][0];
        out[1] = x[i][1];
      }
    }
  }
  if (pe_live) {
    uint4* out = reinterpret_cast<uint4*>(a.k_pe + (row0 + pe_row) * a.k_pe_stride);
    if (kCacheE4m3)
      store_widened(out + 2 * piece, pe, a.k_scale);
    else
      out[piece] = pe;
  }
  if constexpr (kOutE4m3) {  // lane 8 b + i: block b of row i
    const int i = lane % 8;
    float scale = a.k_scale;
    bool live = false;
#pragma unroll
    for (int k = 0; k < kGatherRows; ++k)
      if (i == k) {
        live = src[k] != nullptr;
        if (!kCacheE4m3) scale = scales[k];
      }
    if (live) a.scales[(lane / 8) * a.scale_stride + row0 + i] = scale;
  }
}

// ------------------------------------------------------------------ merge

struct MergeArgs {
  const uint16_t* a;
  const uint16_t* b;
  uint16_t* out;
  const float* lse_a;
  const float* lse_b;
  float* lse;
  int64_t a_ts, a_hs, b_ts, b_hs, o_ts, o_hs;
  int64_t rows;
  int32_t heads, chunks;  // 16-byte pieces of a row
  int32_t block_rows;
};

// A thread merges 8 columns of a row; a block owns whole rows, whose old lse every
// thread reads before the new one is written (they may be the same array).  Bound by
// its bytes: 8192 rows of 128 heads and 128 columns, 818 MB, 125 us (98% of a
// measured copy's rate).
__global__ void __launch_bounds__(kThreads) merge_kernel(const MergeArgs m) {
  grid_dependency();
  const int sub = threadIdx.x / m.chunks, chunk = threadIdx.x - sub * m.chunks;
  const int64_t row = (int64_t)blockIdx.x * m.block_rows + sub;
  const bool live = sub < m.block_rows && row < m.rows;
  float lse = 0.f;
  if (live) {
    const int64_t t = row / m.heads;
    const int h = (int)(row - t * m.heads);
    const uint4 xa = *reinterpret_cast<const uint4*>(m.a + t * m.a_ts + h * m.a_hs + 8 * chunk);
    const uint4 xb = *reinterpret_cast<const uint4*>(m.b + t * m.b_ts + h * m.b_hs + 8 * chunk);
    const float la = m.lse_a[row], lb = m.lse_b[row];
    const float top = fmaxf(la, lb), base = top == -CUDART_INF_F ? 0.f : top;
    // a part without a key may hold anything (its bits are cleared: a branch would put its
    // load behind that of its lse, 142 us for 129)
    const uint32_t keep_a = la == -CUDART_INF_F ? 0u : ~0u, keep_b = lb == -CUDART_INF_F ? 0u : ~0u;
    float wa = __expf(la - base), wb = __expf(lb - base);
    const float sum = wa + wb;
    lse = sum == 0.f ? -CUDART_INF_F : base + logf(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    wa *= inv;
    wb *= inv;
    const uint32_t ua[4] = {xa.x, xa.y, xa.z, xa.w}, ub[4] = {xb.x, xb.y, xb.z, xb.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = ua[i] & keep_a, y = ub[i] & keep_b;
      o[i] = bf16x2(wa * bf_lo(x) + wb * bf_lo(y), wa * bf_hi(x) + wb * bf_hi(y));
    }
    *reinterpret_cast<uint4*>(m.out + t * m.o_ts + h * m.o_hs + 8 * chunk) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  __syncthreads();
  if (live && chunk == 0) m.lse[row] = lse;
}

template <class Kernel, class A>
static cudaError_t launch_pdl(Kernel kernel, int64_t blocks, int threads, cudaStream_t stream, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

static bool multiple(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace mla_pr

// Arguments of every launcher are checked by the caller.
namespace mla {

cudaError_t launch_rope_table(float* table, int64_t first, int64_t positions, int half, const uint64_t* turns,
                              float magnitude, Device dev, cudaStream_t stream) {
  using namespace mla_pr;
  TableArgs a{};
  a.table = table;
  a.first = first;
  a.positions = positions;
  a.half = half;
  a.magnitude = magnitude;
  std::copy(turns, turns + half, a.turns);
  const bool wide = half % 4 == 0 && multiple(table, 16);
  a.block_rows = kThreads / (wide ? half / 4 : half);
  const int64_t singles = (positions + a.block_rows - 1) / a.block_rows, fours = (positions + 4 * a.block_rows - 1) / (4 * a.block_rows);
  if (fours >= dev.sms)
    return wide ? launch_pdl(rope_table_kernel<true, 4>, fours, kThreads, stream, a)
                : launch_pdl(rope_table_kernel<false, 4>, fours, kThreads, stream, a);
  return wide ? launch_pdl(rope_table_kernel<true, 1>, singles, kThreads, stream, a)
              : launch_pdl(rope_table_kernel<false, 1>, singles, kThreads, stream, a);
}

cudaError_t launch_rope(HeadRows q, HeadRows k, HeadRows q_out, HeadRows k_out, const int64_t* positions,
                        const float* table, int64_t max_position, int tokens, int heads, int half, bool neox,
                        cudaStream_t stream) {
  using namespace mla_pr;
  RopeArgs a;
  a.q = static_cast<const uint16_t*>(q.p);
  a.k = static_cast<const uint16_t*>(k.p);
  a.q_out = static_cast<uint16_t*>(const_cast<void*>(q_out.p));
  a.k_out = static_cast<uint16_t*>(const_cast<void*>(k_out.p));
  a.q_ts = q.token_stride;
  a.q_hs = q.head_stride;
  a.qo_ts = q_out.token_stride;
  a.qo_hs = q_out.head_stride;
  a.k_ts = k.token_stride;
  a.ko_ts = k_out.token_stride;
  a.positions = positions;
  a.table = table;
  a.max_position = max_position;
  a.tokens = tokens;
  a.heads = heads;
  a.half = half;
  auto in_pieces = [](const HeadRows& r) {
    return !r.p || (multiple(r.p, 16) && r.token_stride % 8 == 0 && r.head_stride % 8 == 0);
  };
  const bool wide = half % 4 == 0 && multiple(table, 16) && in_pieces(q) && in_pieces(k) && in_pieces(q_out) && in_pieces(k_out);
  a.chunks = wide ? half / 4 : half;
  const int threads = a.chunks <= kRopeThreads ? kRopeThreads : kThreads;  // (a chunk each at least)
  const int slots = threads / a.chunks;
  a.lanes = std::max(1, std::min(slots, heads));
  a.block_tokens = slots / a.lanes;
  const int64_t blocks = ((int64_t)tokens + a.block_tokens - 1) / a.block_tokens;
  if (neox)
    return wide ? launch_pdl(rope_kernel<true, true>, blocks, threads, stream, a) : launch_pdl(rope_kernel<false, true>, blocks, threads, stream, a);
  return wide ? launch_pdl(rope_kernel<true, false>, blocks, threads, stream, a) : launch_pdl(rope_kernel<false, false>, blocks, threads, stream, a);
}

cudaError_t launch_cache_gather(const void* kv, bool kv_e4m3, int64_t num_pages, int page_size, const int32_t* block_table,
                                int64_t bt_stride, const int32_t* starts, const int32_t* cu, int batch, int tokens,
                                float k_scale, void* latent, bool latent_e4m3, int64_t latent_stride, float* scales,
                                int64_t scale_stride, void* k_pe, int64_t k_pe_stride, cudaStream_t stream) {
  using namespace mla_pr;
  GatherArgs a;
  a.kv = static_cast<const uint8_t*>(kv);
  a.block_table = block_table;
  a.starts = starts;
  a.cu = cu;
  a.latent = static_cast<uint8_t*>(latent);
  a.scales = scales;
  a.k_pe = static_cast<uint16_t*>(k_pe);
  a.num_pages = num_pages;
  a.bt_stride = bt_stride;
  a.latent_stride = latent_stride;
  a.scale_stride = scale_stride;
  a.k_pe_stride = k_pe_stride;
  a.page_shift = page_size == 32 ? 5 : 6;
  a.batch = batch;
  a.tokens = tokens;
  a.k_scale = k_scale;
  constexpr int kBlockRows = kGatherThreads / 32 * kGatherRows;
  const int64_t blocks = ((int64_t)tokens + kBlockRows - 1) / kBlockRows;
  if (kv_e4m3)
    return latent_e4m3 ? launch_pdl(cache_gather_kernel<true, true>, blocks, kGatherThreads, stream, a)
                       : launch_pdl(cache_gather_kernel<true, false>, blocks, kGatherThreads, stream, a);
  return latent_e4m3 ? launch_pdl(cache_gather_kernel<false, true>, blocks, kGatherThreads, stream, a)
                     : launch_pdl(cache_gather_kernel<false, false>, blocks, kGatherThreads, stream, a);
}

cudaError_t launch_merge_states(HeadRows x, const float* lse_x, HeadRows y, const float* lse_y, HeadRows out, float* lse,
                                int tokens, int heads, int dim, cudaStream_t stream) {
  using namespace mla_pr;
  MergeArgs m;
  m.a = static_cast<const uint16_t*>(x.p);
  m.b = static_cast<const uint16_t*>(y.p);
  m.out = static_cast<uint16_t*>(const_cast<void*>(out.p));
  m.lse_a = lse_x;
  m.lse_b = lse_y;
  m.lse = lse;
  m.a_ts = x.token_stride;
  m.a_hs = x.head_stride;
  m.b_ts = y.token_stride;
  m.b_hs = y.head_stride;
  m.o_ts = out.token_stride;
  m.o_hs = out.head_stride;
  m.rows = (int64_t)tokens * heads;
  m.heads = heads;
  m.chunks = dim / 8;
  m.block_rows = kThreads / m.chunks;
  return launch_pdl(merge_kernel, (m.rows + m.block_rows - 1) / m.block_rows, kThreads, stream, m);
}

cudaError_t prompt_rows_read_error(int* code, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(code, mla_pr::g_rows_error, sizeof(int));
  if (e != cudaSuccess || !reset) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(mla_pr::g_rows_error, &zero, sizeof(int));
}

}  // namespace mla
