// The row operators of an FP8 layer: RMS norm with the residual's addition,
// and activation quantisation.  Both end in the same quantiser, an e4m3 code
// per element and one fp32 scale for each 128 columns of a row, in the layout
// the FP8 products read.
//
//   add_rmsnorm   h = x + r (fp32), residual_out = round(h),
//                 y = h * rsqrt(mean(h^2) + eps) * weight
//   act_quantize  v = x, or g / (1 + e^-g) * u for a row [g | u]
//   quantiser     s = max(amax |v|, 1e-10) / 448,  code = e4m3(v * (1 / s))
//
// Work item = 8 columns of one row (a 16-byte load); the 16 items of a
// 128-column block sit in 16 neighbouring lanes, so a block's maximum is four
// shuffles.  Maxima are taken on the bit patterns of |v|: patterns order like
// the values with NaN above infinity, so a NaN gives a NaN scale and NaN codes
// instead of being dropped.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/mla_decode.h"

namespace mla_nq {

constexpr float kAmaxFloor = 1e-10f;
constexpr float kE4m3Max = 448.0f;

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// two floats -> two e4m3 bytes, `lo` at the lower address (nearest even, NaN -> NaN)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// g / (1 + e^-g) from e = e^-|g|, which cannot overflow (e^-g does below -88,
// where the result is still a normal number); -inf gives NaN, as the formula.
// 1 + e is in [1, 2]: the quotient by an approximate reciprocal, with one step of
// residual correction, n / d = q + r (n - d q); a residual that is NaN because the
// gate is infinite is bounded and so leaves the quotient as it is.  Within 3 ulp:
// an error here moves codes across rounding borders (with __expf and the bare
// approximation, 6 ulp, twice as many; 10 % faster).
__device__ __forceinline__ float silu(float g) {
  const float e = expf(-fabsf(g)), d = 1.0f + e;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  const float n = g < 0.f ? g * e : g, q = n * r;
  return fmaf(r, fmaxf(fmaf(-d, q, n), -FLT_MAX), q);
}

// Programmatic dependent launch: this kernel may be scheduled while the one
// before it in the stream drains; it touches memory only after that one is
// complete, and lets the next one be scheduled in the same way.
__device__ __forceinline__ void pdl_sync() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A lane's part of a 128-column block of one row: kLanes lanes share the block,
// lane l holds 128 / kLanes columns of it.  kVec: consecutive ones, by 16-byte
// accesses (the row's width is a multiple of 8, so pieces of 8 are whole);
// otherwise columns l, l + kLanes, ..., one by one, so that the lanes' accesses
// still fall into the same sectors (an unaligned row read as 8 neighbours per
// lane took 3.5 times as long).  nb: columns the block has (<= 0: none); absent
// columns read as 0 and are not stored.
template <bool kVec, int kLanes>
__device__ __forceinline__ int column(int l, int k) {
  return kVec ? l * (128 / kLanes) + k : l + kLanes * k;
}
template <bool kVec, int kLanes>
__device__ __forceinline__ void load_bf16(const uint16_t* p, int l, int nb, float (&v)[128 / kLanes]) {
#pragma unroll
  for (int k = 0; k < 128 / kLanes; ++k) v[k] = 0.f;
  if (kVec) {
#pragma unroll
    for (int c = 0; c < 128 / kLanes; c += 8)
      if (column<kVec, kLanes>(l, c) < nb) {
        const uint4 r = *reinterpret_cast<const uint4*>(p + column<kVec, kLanes>(l, c));
        v[c] = bf_lo(r.x); v[c + 1] = bf_hi(r.x); v[c + 2] = bf_lo(r.y); v[c + 3] = bf_hi(r.y);
        v[c + 4] = bf_lo(r.z); v[c + 5] = bf_hi(r.z); v[c + 6] = bf_lo(r.w); v[c + 7] = bf_hi(r.w);
      }
  } else {
#pragma unroll
    for (int k = 0; k < 128 / kLanes; ++k)
      if (column<kVec, kLanes>(l, k) < nb) v[k] = __uint_as_float((uint32_t)p[column<kVec, kLanes>(l, k)] << 16);
  }
}
template <bool kVec, int kLanes>
__device__ __forceinline__ void load_f32(const float* p, int l, int nb, float (&v)[128 / kLanes]) {
#pragma unroll
  for (int k = 0; k < 128 / kLanes; ++k) v[k] = 0.f;
  if (kVec) {
#pragma unroll
    for (int c = 0; c < 128 / kLanes; c += 4)
      if (column<kVec, kLanes>(l, c) < nb) {
        const float4 r = *reinterpret_cast<const float4*>(p + column<kVec, kLanes>(l, c));
        v[c] = r.x; v[c + 1] = r.y; v[c + 2] = r.z; v[c + 3] = r.w;
      }
  } else {
#pragma unroll
    for (int k = 0; k < 128 / kLanes; ++k)
      if (column<kVec, kLanes>(l, k) < nb) v[k] = p[column<kVec, kLanes>(l, k)];
  }
}
template <bool kVec, int kLanes>
__device__ __forceinline__ void store_bf16(uint16_t* p, int l, int nb, const float (&v)[128 / kLanes]) {
  if (kVec) {
#pragma unroll
    for (int c = 0; c < 128 / kLanes; c += 8)
      if (column<kVec, kLanes>(l, c) < nb)
        *reinterpret_cast<uint4*>(p + column<kVec, kLanes>(l, c)) =
            make_uint4(bf16x2(v[c], v[c + 1]), bf16x2(v[c + 2], v[c + 3]), bf16x2(v[c + 4], v[c + 5]),
                       bf16x2(v[c + 6], v[c + 7]));
  } else {
#pragma unroll
    for (int k = 0; k < 128 / kLanes; ++k)
      if (column<kVec, kLanes>(l, k) < nb)
        p[column<kVec, kLanes>(l, k)] = __bfloat16_as_ushort(__float2bfloat16_rn(v[k]));
  }
}
template <bool kVec, int kLanes>
__device__ __forceinline__ void store_f32(float* p, int l, int nb, const float (&v)[128 / kLanes]) {
  if (kVec) {
#pragma unroll
    for (int c = 0; c < 128 / kLanes; c += 4)
      if (column<kVec, kLanes>(l, c) < nb)
        *reinterpret_cast<float4*>(p + column<kVec, kLanes>(l, c)) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < 128 / kLanes; ++k)
      if (column<kVec, kLanes>(l, k) < nb) p[column<kVec, kLanes>(l, k)] = v[k];
  }
}

// The quantiser, run by the kLanes lanes of one 128-column block together (every
// lane of the warp calls it; absent columns are 0 in v).
template <bool kVec, int kLanes>
__device__ __forceinline__ void quantize_block(const float (&v)[128 / kLanes], int l, int nb, uint8_t* dst,
                                               float* scale_dst) {
  constexpr int kN = 128 / kLanes;
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kN; ++k) m = max(m, __float_as_uint(v[k]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float amax = __uint_as_float(m);
  const float scale = __fdiv_rn(amax < kAmaxFloor ? kAmaxFloor : amax, kE4m3Max);  // NaN stays NaN
  const float inv = __frcp_rn(scale);
  if (nb <= 0) return;
  uint32_t w[kN / 4];
#pragma unroll
  for (int k = 0; k < kN / 4; ++k)
    w[k] = e4m3x2(__fmul_rn(v[4 * k], inv), __fmul_rn(v[4 * k + 1], inv)) |
           e4m3x2(__fmul_rn(v[4 * k + 2], inv), __fmul_rn(v[4 * k + 3], inv)) << 16;
  if (kVec) {
#pragma unroll
    for (int c = 0; c < kN; c += 8)
      if (column<kVec, kLanes>(l, c) < nb)
        *reinterpret_cast<uint2*>(dst + column<kVec, kLanes>(l, c)) = make_uint2(w[c / 4], w[c / 4 + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < kN; ++k)
      if (column<kVec, kLanes>(l, k) < nb) dst[column<kVec, kLanes>(l, k)] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
  }
  if (l == 0) *scale_dst = scale;
}

struct NormArgs {
  const uint16_t* x;
  const void* res_in;  // nullptr: no residual
  void* res_out;
  const uint16_t* weight;
  void* y;
  float* y_scales;  // [blocks][scale_stride] (e4m3 output)
  int64_t x_stride, res_stride, y_stride, scale_stride;
  int num_tokens, dim;
  float eps;
};

constexpr int kRowsPerCta = 4;  // of the form with a warp per row

// One CTA per row, or (kWarpRow, rows up to 1024 columns) one warp per row: the
// row stays in registers (kChunks pieces of 8 columns per thread) between the
// sum of squares and the output, so every input byte is read once.  A CTA per
// row spends more on scheduling than on a narrow row: 16384 rows of 512 take
// 17 us by CTAs.  kRes: 0 none, 1 bf16, 2 fp32.
template <int kChunks, bool kVec, int kRes, bool kE4m3, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowsPerCta : 1024) add_rmsnorm_kernel(const NormArgs a) {
  pdl_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = kWarpRow ? (int64_t)blockIdx.x * kRowsPerCta + warp : blockIdx.x;
  if (kWarpRow && t >= a.num_tokens) return;
  const int first = kWarpRow ? lane : threadIdx.x, step = kWarpRow ? 32 : blockDim.x;
  const int l = lane & 15;  // 16 lanes to a 128-column block
  __shared__ float part[32];
  float h[kChunks][8];
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = ((first + c * step) >> 4) * 128, nb = a.dim - col;
    load_bf16<kVec, 16>(a.x + t * a.x_stride + col, l, nb, h[c]);
    if (kRes != 0) {
      float r[8];
      const int64_t at = t * a.res_stride + col;
      if (kRes == 1)
        load_bf16<kVec, 16>(static_cast<const uint16_t*>(a.res_in) + at, l, nb, r);
      else
        load_f32<kVec, 16>(static_cast<const float*>(a.res_in) + at, l, nb, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] += r[i];
      if (kRes == 1)
        store_bf16<kVec, 16>(static_cast<uint16_t*>(a.res_out) + at, l, nb, h[c]);
      else
        store_f32<kVec, 16>(static_cast<float*>(a.res_out) + at, l, nb, h[c]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);  // absent columns are 0
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (!kWarpRow) {
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    sum = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const float rstd = rsqrtf(sum / (float)a.dim + a.eps);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int block = (first + c * step) >> 4, nb = a.dim - 128 * block;
    float w[8];
    load_bf16<kVec, 16>(a.weight + 128 * block, l, nb, w);
    // absent columns stay 0 (0 * NaN would reach the block's maximum)
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] = column<kVec, 16>(l, i) < nb ? h[c][i] * rstd * w[i] : 0.f;
    if (kE4m3)
      quantize_block<kVec, 16>(h[c], l, nb, static_cast<uint8_t*>(a.y) + t * a.y_stride + 128 * block,
                               a.y_scales + (int64_t)block * a.scale_stride + t);
    else
      store_bf16<kVec, 16>(static_cast<uint16_t*>(a.y) + t * a.y_stride + 128 * block, l, nb, h[c]);
  }
}

// Many wide rows: persistent CTAs that fetch the next row's inputs before they
// reduce the current one, so that loads are in flight throughout (a CTA per row
// loads, waits and stores in turn: 16384 x 8192 with residual 168 us).  Whole
// 16-byte pieces, kRowsChunks of them per thread; the weights stay in registers.
// kRes: a bf16 residual.
constexpr int kRowsChunks = 2, kRowsThreads = 512;
template <bool kRes, bool kE4m3>
__global__ void __launch_bounds__(kRowsThreads, 2) add_rmsnorm_rows_kernel(const NormArgs a) {
  pdl_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 15;
  __shared__ float part[2][32];
  uint4 px[kRowsChunks], pr[kRowsChunks], pw[kRowsChunks];
  auto col_of = [&](int c) { return 8 * (int)(threadIdx.x + c * blockDim.x); };
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int c = 0; c < kRowsChunks; ++c) {
      const int col = col_of(c);
      if (col < a.dim) {
        px[c] = *reinterpret_cast<const uint4*>(a.x + t * a.x_stride + col);
        if (kRes) pr[c] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.res_in) + t * a.res_stride + col);
      }
    }
  };
  auto unpack = [](uint4 r, float (&v)[8]) {
    v[0] = bf_lo(r.x); v[1] = bf_hi(r.x); v[2] = bf_lo(r.y); v[3] = bf_hi(r.y);
    v[4] = bf_lo(r.z); v[5] = bf_hi(r.z); v[6] = bf_lo(r.w); v[7] = bf_hi(r.w);
  };
#pragma unroll
  for (int c = 0; c < kRowsChunks; ++c) {
    px[c] = pr[c] = pw[c] = make_uint4(0u, 0u, 0u, 0u);  // absent columns stay 0
    if (col_of(c) < a.dim) pw[c] = *reinterpret_cast<const uint4*>(a.weight + col_of(c));
  }
  int64_t t = blockIdx.x;
  fetch(t);
  for (int turn = 0; t < a.num_tokens; turn ^= 1) {
    float h[kRowsChunks][8];
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < kRowsChunks; ++c) {
      const int col = col_of(c);
      unpack(px[c], h[c]);
      if (kRes) {
        float r[8];
        unpack(pr[c], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += r[i];
        if (col < a.dim) store_bf16<true, 16>(static_cast<uint16_t*>(a.res_out) + t * a.res_stride + col, 0, 8, h[c]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
    }
    const int64_t now = t;
    t += gridDim.x;
    if (t < a.num_tokens) fetch(t);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[turn][warp] = sum;
    __syncthreads();  // one per row: the next row's partial sums go to the other half
    sum = lane < (int)(blockDim.x >> 5) ? part[turn][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float rstd = rsqrtf(sum / (float)a.dim + a.eps);
#pragma unroll
    for (int c = 0; c < kRowsChunks; ++c) {
      const int col = col_of(c), block = col >> 7, nb = a.dim - 128 * block;
      float w[8];
      unpack(pw[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = col < a.dim ? h[c][i] * rstd * w[i] : 0.f;
      if (kE4m3)
        quantize_block<true, 16>(h[c], l, nb, static_cast<uint8_t*>(a.y) + now * a.y_stride + 128 * block,
                                 a.y_scales + (int64_t)block * a.scale_stride + now);
      else
        store_bf16<true, 16>(static_cast<uint16_t*>(a.y) + now * a.y_stride + 128 * block, l, nb, h[c]);
    }
  }
}

struct ActArgs {
  const uint16_t* x;
  void* y;
  float* y_scales;
  int64_t x_stride, y_stride, scale_stride;
  int num_tokens, dim;
  int row_shift;  // log2 of the lanes that share a row: 3, 4 or 5 (128, 256 or 512 columns)
};

constexpr int kActThreads = 256;

// A lane takes 16 columns (two 16-byte loads per operand), 8 lanes a 128-column
// block.  A CTA takes consecutive rows of one 512-column segment (narrow rows:
// several rows per warp), so that the scales of neighbouring tokens are stored
// together and no index is divided.
template <bool kVec, bool kSiluMul, bool kE4m3>
__global__ void __launch_bounds__(kActThreads) act_quantize_kernel(const ActArgs a) {
  pdl_sync();
  const int64_t t = ((int64_t)blockIdx.x * kActThreads + threadIdx.x) >> a.row_shift;
  const int l = threadIdx.x & 7;
  const int block = ((blockIdx.y << a.row_shift) + (threadIdx.x & ((1 << a.row_shift) - 1))) >> 3;
  const int nb = t < a.num_tokens ? a.dim - 128 * block : 0;
  const uint16_t* x = a.x + t * a.x_stride + 128 * block;
  float v[16];
  load_bf16<kVec, 8>(x, l, nb, v);
  if (kSiluMul) {
    float u[16];
    load_bf16<kVec, 8>(x + a.dim, l, nb, u);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = silu(v[i]) * u[i];  // absent columns: 0
  }
  if (kE4m3)
    quantize_block<kVec, 8>(v, l, nb, static_cast<uint8_t*>(a.y) + t * a.y_stride + 128 * block,
                            a.y_scales + (int64_t)block * a.scale_stride + t);
  else
    store_bf16<kVec, 8>(static_cast<uint16_t*>(a.y) + t * a.y_stride + 128 * block, l, nb, v);
}

template <class Kernel, class A>
static cudaError_t launch_pdl(Kernel kernel, dim3 blocks, unsigned threads, cudaStream_t stream, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = blocks;
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

template <int kChunks, bool kVec, int kRes, bool kWarpRow>
static cudaError_t launch_norm_out(const NormArgs& a, int threads, bool e4m3, cudaStream_t stream) {
  const dim3 grid(kWarpRow ? (unsigned)(((int64_t)a.num_tokens + kRowsPerCta - 1) / kRowsPerCta) : a.num_tokens);
  return e4m3 ? launch_pdl(add_rmsnorm_kernel<kChunks, kVec, kRes, true, kWarpRow>, grid, threads, stream, a)
              : launch_pdl(add_rmsnorm_kernel<kChunks, kVec, kRes, false, kWarpRow>, grid, threads, stream, a);
}

template <int kChunks, bool kWarpRow, bool kVec>
static cudaError_t launch_norm_res(const NormArgs& a, int threads, int res, bool e4m3, cudaStream_t stream) {
  if (res == 0) return launch_norm_out<kChunks, kVec, 0, kWarpRow>(a, threads, e4m3, stream);
  if (res == 1) return launch_norm_out<kChunks, kVec, 1, kWarpRow>(a, threads, e4m3, stream);
  return launch_norm_out<kChunks, kVec, 2, kWarpRow>(a, threads, e4m3, stream);
}

template <bool kRes>
static cudaError_t launch_norm_rows(const NormArgs& a, int items, bool e4m3, int sms, cudaStream_t stream) {
  const int threads = ((items + kRowsChunks - 1) / kRowsChunks + 31) / 32 * 32;
  const dim3 grid(std::min(a.num_tokens, sms * std::max(1, 2 * kRowsThreads / threads)));
  return e4m3 ? launch_pdl(add_rmsnorm_rows_kernel<kRes, true>, grid, threads, stream, a)
              : launch_pdl(add_rmsnorm_rows_kernel<kRes, false>, grid, threads, stream, a);
}

template <int kChunks, bool kWarpRow>
static cudaError_t launch_norm(const NormArgs& a, int items, bool vec, int res, bool e4m3, cudaStream_t stream) {
  const int threads = kWarpRow ? 32 * kRowsPerCta : ((items + kChunks - 1) / kChunks + 31) / 32 * 32;
  return vec ? launch_norm_res<kChunks, kWarpRow, true>(a, threads, res, e4m3, stream)
             : launch_norm_res<kChunks, kWarpRow, false>(a, threads, res, e4m3, stream);
}

}  // namespace mla_nq

namespace mla {

// residual_kind: 0 none, 1 bf16, 2 fp32.  Arguments are checked by the caller.
cudaError_t launch_add_rmsnorm(const void* x, int64_t x_stride, const void* res_in, void* res_out, int residual_kind,
                               int64_t res_stride, const void* weight, int num_tokens, int dim, float eps, void* y,
                               int64_t y_stride, bool e4m3, float* y_scales, int64_t scale_stride, int sms,
                               cudaStream_t stream) {
  using namespace mla_nq;
  NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.res_in = res_in;
  a.res_out = res_out;
  a.weight = static_cast<const uint16_t*>(weight);
  a.y = y;
  a.y_scales = y_scales;
  a.x_stride = x_stride;
  a.res_stride = res_stride;
  a.y_stride = y_stride;
  a.scale_stride = scale_stride;
  a.num_tokens = num_tokens;
  a.dim = dim;
  a.eps = eps;
  // 16-byte accesses need every row to start on their boundary; anything else
  // takes the element-wise form of the same kernel
  const bool vec = dim % 8 == 0 && x_stride % 8 == 0 && y_stride % 8 == 0 && multiple(x, 16) && multiple(weight, 16) &&
                   multiple(y, e4m3 ? 8 : 16) &&
                   (residual_kind == 0 ||
                    (res_stride % 8 == 0 && multiple(res_in, 16) && multiple(res_out, 16)));
  const int items = (dim + 127) / 128 * 16;  // 8-column pieces of whole blocks
  // Rows enough to stay busy: persistent CTAs (16384 x 8192 with a bf16 residual
  // 153 us against 168 by a CTA per row, 16384 x 4096 without one 42 against 49).
  // Not with an fp32 residual, whose wider fetches cost more registers than they
  // win (130 against 107).
  if (vec && residual_kind != 2 && items > 128 && items <= kRowsChunks * kRowsThreads && num_tokens >= 4 * sms)
    return residual_kind == 0 ? launch_norm_rows<false>(a, items, e4m3, sms, stream)
                              : launch_norm_rows<true>(a, items, e4m3, sms, stream);
  if (items <= 32) return launch_norm<1, true>(a, items, vec, residual_kind, e4m3, stream);
  if (items <= 64) return launch_norm<2, true>(a, items, vec, residual_kind, e4m3, stream);
  if (items <= 128) return launch_norm<4, true>(a, items, vec, residual_kind, e4m3, stream);
  if (items <= 1024) return launch_norm<1, false>(a, items, vec, residual_kind, e4m3, stream);
  if (items <= 2048) return launch_norm<2, false>(a, items, vec, residual_kind, e4m3, stream);
  return launch_norm<4, false>(a, items, vec, residual_kind, e4m3, stream);
}

cudaError_t launch_act_quantize(const void* x, int64_t x_stride, int num_tokens, int dim, bool silu_mul, void* y,
                                int64_t y_stride, bool e4m3, float* y_scales, int64_t scale_stride,
                                cudaStream_t stream) {
  using namespace mla_nq;
  ActArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.y = y;
  a.y_scales = y_scales;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.scale_stride = scale_stride;
  a.num_tokens = num_tokens;
  a.dim = dim;
  a.row_shift = dim <= 128 ? 3 : dim <= 256 ? 4 : 5;
  const bool vec = dim % 8 == 0 && x_stride % 8 == 0 && y_stride % 8 == 0 && multiple(x, 16) && multiple(y, e4m3 ? 8 : 16);
  const int rows = kActThreads >> a.row_shift, cols = 16 << a.row_shift;
  const dim3 blocks((unsigned)(((int64_t)num_tokens + rows - 1) / rows), (unsigned)(((int64_t)dim + cols - 1) / cols));
  if (silu_mul && e4m3)
    return vec ? launch_pdl(act_quantize_kernel<true, true, true>, blocks, kActThreads, stream, a)
               : launch_pdl(act_quantize_kernel<false, true, true>, blocks, kActThreads, stream, a);
  if (silu_mul)
    return vec ? launch_pdl(act_quantize_kernel<true, true, false>, blocks, kActThreads, stream, a)
               : launch_pdl(act_quantize_kernel<false, true, false>, blocks, kActThreads, stream, a);
  return vec ? launch_pdl(act_quantize_kernel<true, false, true>, blocks, kActThreads, stream, a)
             : launch_pdl(act_quantize_kernel<false, false, true>, blocks, kActThreads, stream, a);
}

}  // namespace mla
