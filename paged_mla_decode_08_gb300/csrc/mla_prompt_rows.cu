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
// in 64 bits and the product taken modulo 2^64, so the reduction costs one integer
// product and is exact to 2^-64 of a turn a position, however far (double
// precision, at this GPU's rate, would be what bounds the kernel).  The upper 24
// bits of the reduced turn are exact in fp32 and go through sincospif; the rest d
// enters as cos - d sin, sin + d cos.
struct TableArgs {
  float* table;
  int64_t first, positions;
  int32_t half;  // pairs of a row
  float magnitude;
  uint64_t turns[MLA_ROPE_MAX_DIM / 2];  // of a position, in 2^-64 of a turn
};

__device__ __forceinline__ void cos_sin(uint64_t turn, float magnitude, float* c, float* s) {
  const int64_t t = static_cast<int64_t>(turn);  // [-1/2, 1/2) of a turn
  const float low = static_cast<float>(static_cast<uint32_t>(turn >> 8)) * (2.f * CUDART_PI_F * 0x1p-56f);
  float c0, s0;
  sincospif(static_cast<float>(static_cast<int32_t>(t >> 40)) * 0x1p-23f, &s0, &c0);
  *c = fmaf(-low, s0, c0) * magnitude;
  *s = fmaf(low, c0, s0) * magnitude;
}

// kWide: four pairs a thread (half % 4 == 0, 16-byte rows); else one
template <bool kWide>
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ TableArgs a) {
  grid_dependency();
  constexpr int kPairs = kWide ? 4 : 1;
  const int per_row = a.half / kPairs;
  const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (item >= a.positions * per_row) return;
  const int64_t p = item / per_row;
  const int i = (int)(item - p * per_row) * kPairs;
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int k = 0; k < kPairs; ++k)
    cos_sin(static_cast<uint64_t>(a.first + p) * a.turns[i + k], a.magnitude, c + k, s + k);
  float* row = a.table + p * 2 * a.half + i;
  if (kWide) {
    *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1 % kPairs], c[2 % kPairs], c[3 % kPairs]);
    *reinterpret_cast<float4*>(row + a.half) = make_float4(s[0], s[1 % kPairs], s[2 % kPairs], s[3 % kPairs]);
  } else {
    row[0] = c[0];
    row[a.half] = s[0];
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
  int32_t tokens, heads;  // heads: query heads; the key is one row more
  int32_t rows;           // of a token: heads, and the key if there is one
  int32_t half, neox;
  int32_t chunks;         // of a row: threads that share it
  int32_t lanes;          // rows of a token at a time
  int32_t block_tokens;   // tokens of a block
};

__device__ __forceinline__ const uint16_t* rope_src(const RopeArgs& a, int64_t t, int h) {
  return h < a.heads ? a.q + t * a.q_ts + h * a.q_hs : a.k + t * a.k_ts;
}
__device__ __forceinline__ uint16_t* rope_dst(const RopeArgs& a, int64_t t, int h) {
  return h < a.heads ? a.q_out + t * a.qo_ts + h * a.qo_hs : a.k_out + t * a.ko_ts;
}

// A thread keeps the cosines and sines of its pairs (four, or one where rows are
// not made of 16-byte pieces) and rotates them in several heads of its token.  Each
// product and sum is rounded to fp32 on its own, as in the cache write's rotation.
template <bool kWide>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  grid_dependency();
  const int chunk = threadIdx.x % a.chunks, slot = threadIdx.x / a.chunks;
  const int sub = slot / a.lanes, lane = slot - sub * a.lanes;
  const int64_t t = (int64_t)blockIdx.x * a.block_tokens + sub;
  if (sub >= a.block_tokens || t >= a.tokens) return;
  const int64_t pos = a.positions[t];
  if (pos < 0 || pos >= a.max_position) {
    if (chunk == 0 && lane == 0) record(0x801);
    return;  // nothing of this token is written
  }
  const float* row = a.table + pos * 2 * a.half;
  if (kWide) {
    const float4 c = *reinterpret_cast<const float4*>(row + 4 * chunk);
    const float4 s = *reinterpret_cast<const float4*>(row + a.half + 4 * chunk);
    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
    auto load = [&](int h) {
      const uint16_t* x = rope_src(a, t, h);
      if (!a.neox) return *reinterpret_cast<const uint4*>(x + 8 * chunk);
      const uint2 lo = *reinterpret_cast<const uint2*>(x + 4 * chunk), hi = *reinterpret_cast<const uint2*>(x + a.half + 4 * chunk);
      return make_uint4(lo.x, lo.y, hi.x, hi.y);
    };
    auto rotate = [&](int h, uint4 v) {
      float x[4], y[4], p[4], q[4];
      if (a.neox) {
        x[0] = bf_lo(v.x); x[1] = bf_hi(v.x); x[2] = bf_lo(v.y); x[3] = bf_hi(v.y);
        y[0] = bf_lo(v.z); y[1] = bf_hi(v.z); y[2] = bf_lo(v.w); y[3] = bf_hi(v.w);
      } else {
        x[0] = bf_lo(v.x); y[0] = bf_hi(v.x); x[1] = bf_lo(v.y); y[1] = bf_hi(v.y);
        x[2] = bf_lo(v.z); y[2] = bf_hi(v.z); x[3] = bf_lo(v.w); y[3] = bf_hi(v.w);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = __fsub_rn(__fmul_rn(x[i], cs[i]), __fmul_rn(y[i], sn[i]));
        q[i] = __fadd_rn(__fmul_rn(y[i], cs[i]), __fmul_rn(x[i], sn[i]));
      }
      uint16_t* o = rope_dst(a, t, h);
      if (a.neox) {
        *reinterpret_cast<uint2*>(o + 4 * chunk) = make_uint2(bf16x2(p[0], p[1]), bf16x2(p[2], p[3]));
        *reinterpret_cast<uint2*>(o + a.half + 4 * chunk) = make_uint2(bf16x2(q[0], q[1]), bf16x2(q[2], q[3]));
      } else {
        *reinterpret_cast<uint4*>(o + 8 * chunk) =
            make_uint4(bf16x2(p[0], q[0]), bf16x2(p[1], q[1]), bf16x2(p[2], q[2]), bf16x2(p[3], q[3]));
      }
    };
    int h = lane;
    for (; h + 3 * a.lanes < a.rows; h += 4 * a.lanes) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = load(h + i * a.lanes);
#pragma unroll
      for (int i = 0; i < 4; ++i) rotate(h + i * a.lanes, v[i]);
    }
    for (; h < a.rows; h += a.lanes) rotate(h, load(h));
  } else {
    const float c = row[chunk], s = row[a.half + chunk];
    const int at0 = a.neox ? chunk : 2 * chunk, at1 = a.neox ? a.half + chunk : 2 * chunk + 1;
    for (int h = lane; h < a.rows; h += a.lanes) {
      const uint16_t* x = rope_src(a, t, h);
      const float u = bf(x[at0]), v = bf(x[at1]);
      uint16_t* o = rope_dst(a, t, h);
      o[at0] = to_bf16(__fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s)));
      o[at1] = to_bf16(__fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s)));
    }
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

constexpr int kGatherRows = 4;  // of a warp

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
    const bool le = lane * step < n && __ldg(a.cu + at) <= r;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    const int end = min(lo + n, lo + (last + 1) * step);
    lo += last * step;
    n = end - lo;
  }
  return lo;
}

// A warp copies four consecutive rows; a lane 16 latent columns and, the first
// ones, a piece of the rotary ones.
template <bool kCacheE4m3, bool kOutE4m3>
__global__ void __launch_bounds__(kThreads) cache_gather_kernel(const GatherArgs a) {
  grid_dependency();
  const int lane = threadIdx.x & 31;
  const int64_t row0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kGatherRows;
  if (blockIdx.x == 0 && threadIdx.x < 32) {  // the offsets' rules, looked at once
    bool bad = false;
    for (int b = lane; b <= a.batch; b += 32) {
      const int c = __ldg(a.cu + b);
      bad |= c < 0 || c > a.tokens || (b > 0 && c < __ldg(a.cu + b - 1));
    }
    if (bad) record(0x903);
  }
  if (row0 >= a.tokens) return;
  constexpr int kRowBytes = kCacheE4m3 ? 576 : 1152, kLaneBytes = kCacheE4m3 ? 16 : 32;
  const int my_row = (int)row0 + min(lane, kGatherRows - 1);
  const uint8_t* src_mine = nullptr;
  {
    int b = owner(a, (int)row0, lane);
    if (lane < kGatherRows && my_row < a.tokens) {
      while (b < a.batch && __ldg(a.cu + b + 1) <= my_row) ++b;
      if (b < a.batch) {
        const int begin = __ldg(a.cu + b);
        const int64_t token = (a.starts ? (int64_t)__ldg(a.starts + b) : 0) + my_row - begin;
        if (my_row >= begin) {
          const int64_t block = token >> a.page_shift;
          if (token < 0 || block >= a.bt_stride) {
            record(0x901);
          } else {
            const int64_t page = __ldg(a.block_table + b * a.bt_stride + block);
            if (page < 0 || page >= a.num_pages)
              record(0x902);
            else
              src_mine = a.kv + ((page << a.page_shift) + (token & ((1 << a.page_shift) - 1))) * kRowBytes;
          }
        }
      }
    }
  }
  const uint8_t* src[kGatherRows];
  uint4 x[kGatherRows][kLaneBytes / 16], pe[kGatherRows];
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    src[i] = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src_mine), i));
    if (src[i]) {
#pragma unroll
      for (int k = 0; k < kLaneBytes / 16; ++k) x[i][k] = *reinterpret_cast<const uint4*>(src[i] + lane * kLaneBytes + 16 * k);
      if (lane < kRowBytes / 144) pe[i] = *reinterpret_cast<const uint4*>(src[i] + 32 * kLaneBytes + 16 * lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    if (!src[i]) continue;
    const int64_t r = row0 + i;
    uint16_t* pe_out = a.k_pe + r * a.k_pe_stride;
    if (kCacheE4m3) {
      if (lane < 4) {
        const uint2 p0 = widen(pe[i].x, a.k_scale), p1 = widen(pe[i].y, a.k_scale), p2 = widen(pe[i].z, a.k_scale),
                    p3 = widen(pe[i].w, a.k_scale);
        reinterpret_cast<uint4*>(pe_out)[2 * lane] = make_uint4(p0.x, p0.y, p1.x, p1.y);
        reinterpret_cast<uint4*>(pe_out)[2 * lane + 1] = make_uint4(p2.x, p2.y, p3.x, p3.y);
      }
    } else if (lane < 8) {
      reinterpret_cast<uint4*>(pe_out)[lane] = pe[i];
    }
    if (kOutE4m3) {
      uint4* out = reinterpret_cast<uint4*>(a.latent + r * a.latent_stride) + lane;
      float scale = a.k_scale;
      if (kCacheE4m3) {
        *out = x[i][0];  // the codes as they are, with the cache's scale
      } else {
        float v[16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 w = x[i][k % (kLaneBytes / 16)];
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
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
        for (int d = 1; d < 8; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));  // a block of 128: 8 lanes
        const float amax = __uint_as_float(top);
        scale = __fdiv_rn(amax < 1e-10f ? 1e-10f : amax, 448.f);
        const float inv = __frcp_rn(scale);
        uint32_t code[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          code[e] = e4m3x2(__fmul_rn(v[4 * e], inv), __fmul_rn(v[4 * e + 1], inv)) |
                    (uint32_t)e4m3x2(__fmul_rn(v[4 * e + 2], inv), __fmul_rn(v[4 * e + 3], inv)) << 16;
        *out = make_uint4(code[0], code[1], code[2], code[3]);
      }
      if (lane % 8 == 0) a.scales[(lane / 8) * a.scale_stride + r] = scale;
    } else {
      uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.latent) + r * a.latent_stride) + 2 * lane;
      if (kCacheE4m3) {
        const uint2 p0 = widen(x[i][0].x, a.k_scale), p1 = widen(x[i][0].y, a.k_scale), p2 = widen(x[i][0].z, a.k_scale),
                    p3 = widen(x[i][0].w, a.k_scale);
        out[0] = make_uint4(p0.x, p0.y, p1.x, p1.y);
        out[1] = make_uint4(p2.x, p2.y, p3.x, p3.y);
      } else {
        out[0] = x[i][0];
        out[1] = x[i][kLaneBytes / 16 - 1];
      }
    }
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
// thread reads before the new one is written (they may be the same array).
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
      // a part that weighs nothing may hold anything
      const float a0 = wa == 0.f ? 0.f : wa * bf_lo(ua[i]), a1 = wa == 0.f ? 0.f : wa * bf_hi(ua[i]);
      const float b0 = wb == 0.f ? 0.f : wb * bf_lo(ub[i]), b1 = wb == 0.f ? 0.f : wb * bf_hi(ub[i]);
      o[i] = bf16x2(a0 + b0, a1 + b1);
    }
    *reinterpret_cast<uint4*>(m.out + t * m.o_ts + h * m.o_hs + 8 * chunk) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  __syncthreads();
  if (live && chunk == 0) m.lse[row] = lse;
}

template <class Kernel, class A>
static cudaError_t launch_pdl(Kernel kernel, int64_t blocks, cudaStream_t stream, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
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
                              float magnitude, cudaStream_t stream) {
  using namespace mla_pr;
  TableArgs a{};
  a.table = table;
  a.first = first;
  a.positions = positions;
  a.half = half;
  a.magnitude = magnitude;
  std::copy(turns, turns + half, a.turns);
  const bool wide = half % 4 == 0 && multiple(table, 16);
  const int64_t items = positions * (wide ? half / 4 : half), blocks = (items + kThreads - 1) / kThreads;
  return wide ? launch_pdl(rope_table_kernel<true>, blocks, stream, a) : launch_pdl(rope_table_kernel<false>, blocks, stream, a);
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
  a.rows = heads + (k.p ? 1 : 0);
  a.half = half;
  a.neox = neox;
  auto in_pieces = [](const HeadRows& r) {
    return !r.p || (multiple(r.p, 16) && r.token_stride % 8 == 0 && r.head_stride % 8 == 0);
  };
  const bool wide = half % 4 == 0 && multiple(table, 16) && in_pieces(q) && in_pieces(k) && in_pieces(q_out) && in_pieces(k_out);
  a.chunks = wide ? half / 4 : half;
  const int slots = kThreads / a.chunks;
  a.lanes = std::min(slots, a.rows);
  a.block_tokens = slots / a.lanes;
  const int64_t blocks = ((int64_t)tokens + a.block_tokens - 1) / a.block_tokens;
  return wide ? launch_pdl(rope_kernel<true>, blocks, stream, a) : launch_pdl(rope_kernel<false>, blocks, stream, a);
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
  constexpr int kBlockRows = kThreads / 32 * kGatherRows;
  const int64_t blocks = ((int64_t)tokens + kBlockRows - 1) / kBlockRows;
  if (kv_e4m3)
    return latent_e4m3 ? launch_pdl(cache_gather_kernel<true, true>, blocks, stream, a)
                       : launch_pdl(cache_gather_kernel<true, false>, blocks, stream, a);
  return latent_e4m3 ? launch_pdl(cache_gather_kernel<false, true>, blocks, stream, a)
                     : launch_pdl(cache_gather_kernel<false, false>, blocks, stream, a);
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
  return launch_pdl(merge_kernel, (m.rows + m.block_rows - 1) / m.block_rows, stream, m);
}

cudaError_t prompt_rows_read_error(int* code, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(code, mla_pr::g_rows_error, sizeof(int));
  if (e != cudaSuccess || !reset) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(mla_pr::g_rows_error, &zero, sizeof(int));
}

}  // namespace mla
