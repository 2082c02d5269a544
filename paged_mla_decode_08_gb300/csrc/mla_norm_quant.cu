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
#include <stdint.h>

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
__device__ __forceinline__ float silu(float g) {
  const float e = __expf(-fabsf(g));
  return g * (g < 0.f ? e : 1.0f) / (1.0f + e);
}

// Programmatic dependent launch: this kernel may be scheduled while the one
// before it in the stream drains; it touches memory only after that one is
// complete, and lets the next one be scheduled in the same way.
__device__ __forceinline__ void pdl_sync() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// 8 consecutive columns of a row.  kVec: 16-byte accesses (all 8 present);
// otherwise element by element, the columns past n reading as 0 and not stored.
template <bool kVec>
__device__ __forceinline__ void load_bf16(const uint16_t* p, int n, float v[8]) {
  if (kVec) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    v[0] = bf_lo(r.x); v[1] = bf_hi(r.x); v[2] = bf_lo(r.y); v[3] = bf_hi(r.y);
    v[4] = bf_lo(r.z); v[5] = bf_hi(r.z); v[6] = bf_lo(r.w); v[7] = bf_hi(r.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __uint_as_float((uint32_t)p[i] << 16) : 0.f;
  }
}
template <bool kVec>
__device__ __forceinline__ void load_f32(const float* p, int n, float v[8]) {
  if (kVec) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}
template <bool kVec>
__device__ __forceinline__ void store_bf16(uint16_t* p, int n, const float v[8]) {
  if (kVec) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
  }
}
template <bool kVec>
__device__ __forceinline__ void store_f32(float* p, int n, const float v[8]) {
  if (kVec) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

// The quantiser, run by the 16 lanes of one 128-column block together (every
// lane of the half warp calls it; n = valid columns of this lane, 0 for none).
template <bool kVec>
__device__ __forceinline__ void quantize_block(const float v[8], int n, uint8_t* dst, float* scale_dst, int lane) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);  // absent columns are 0
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float amax = __uint_as_float(m);
  const float scale = __fdiv_rn(amax < kAmaxFloor ? kAmaxFloor : amax, kE4m3Max);  // NaN stays NaN
  const float inv = __fdiv_rn(1.0f, scale);
  if (n > 0) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e4m3x2(__fmul_rn(v[2 * i], inv), __fmul_rn(v[2 * i + 1], inv));
    if (kVec) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) dst[i] = (uint8_t)(w[i >> 1] >> (8 * (i & 1)));
    }
    if ((lane & 15) == 0) *scale_dst = scale;
  }
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

// One CTA per row: the row stays in registers (kChunks items per thread)
// between the sum of squares and the output, so every input byte is read once.
// kRes: 0 none, 1 bf16, 2 fp32.
template <int kChunks, bool kVec, int kRes, bool kE4m3>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const NormArgs a) {
  pdl_sync();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ float part[32];
  float h[kChunks][8];
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = 8 * (threadIdx.x + c * blockDim.x);
    const int n = min(8, a.dim - col);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] = 0.f;
    if (n > 0) {
      load_bf16<kVec>(a.x + t * a.x_stride + col, n, h[c]);
      if (kRes != 0) {
        float r[8];
        if (kRes == 1)
          load_bf16<kVec>(static_cast<const uint16_t*>(a.res_in) + t * a.res_stride + col, n, r);
        else
          load_f32<kVec>(static_cast<const float*>(a.res_in) + t * a.res_stride + col, n, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += r[i];
        if (kRes == 1)
          store_bf16<kVec>(static_cast<uint16_t*>(a.res_out) + t * a.res_stride + col, n, h[c]);
        else
          store_f32<kVec>(static_cast<float*>(a.res_out) + t * a.res_stride + col, n, h[c]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  sum = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float rstd = rsqrtf(sum / (float)a.dim + a.eps);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = 8 * (threadIdx.x + c * blockDim.x);
    const int n = min(8, a.dim - col);
    float w[8];
    if (n > 0) {
      load_bf16<kVec>(a.weight + col, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * rstd * (kVec || i < n ? w[i] : 0.f);
    }
    if (kE4m3) {
      // absent columns must not reach the maximum (0 * NaN would)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = i < n ? h[c][i] : 0.f;
      quantize_block<kVec>(h[c], n, static_cast<uint8_t*>(a.y) + t * a.y_stride + col,
                           a.y_scales + (int64_t)(col >> 7) * a.scale_stride + t, lane);
    } else if (n > 0) {
      store_bf16<kVec>(static_cast<uint16_t*>(a.y) + t * a.y_stride + col, n, h[c]);
    }
  }
}

struct ActArgs {
  const uint16_t* x;
  void* y;
  float* y_scales;
  int64_t x_stride, y_stride, scale_stride;
  int64_t items;  // num_tokens * items_per_row
  int dim, items_per_row;
};

constexpr int kActThreads = 256;

// One thread per item over a flat grid; items_per_row is a multiple of 16, so
// a block's 16 items are 16 neighbouring lanes.
template <bool kVec, bool kSiluMul, bool kE4m3>
__global__ void __launch_bounds__(kActThreads) act_quantize_kernel(const ActArgs a) {
  pdl_sync();
  const int64_t item = (int64_t)blockIdx.x * kActThreads + threadIdx.x;
  const bool live = item < a.items;  // whole half warps: items is a multiple of 16
  const int64_t t = live ? item / a.items_per_row : 0;
  const int col = 8 * (int)(live ? item - t * a.items_per_row : 0);
  const int n = live ? min(8, a.dim - col) : 0;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (n > 0) {
    load_bf16<kVec>(a.x + t * a.x_stride + col, n, v);
    if (kSiluMul) {
      float u[8];
      load_bf16<kVec>(a.x + t * a.x_stride + a.dim + col, n, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = silu(v[i]) * u[i];
    }
  }
  if (kE4m3)
    quantize_block<kVec>(v, n, static_cast<uint8_t*>(a.y) + t * a.y_stride + col,
                         a.y_scales + (int64_t)(col >> 7) * a.scale_stride + t, threadIdx.x & 31);
  else if (n > 0)
    store_bf16<kVec>(static_cast<uint16_t*>(a.y) + t * a.y_stride + col, n, v);
}

template <class Kernel, class A>
static void launch_pdl(Kernel kernel, unsigned blocks, unsigned threads, cudaStream_t stream, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, a);  // an error is read with cudaGetLastError
}

static bool multiple(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int kChunks, bool kVec, int kRes>
static void launch_norm_out(const NormArgs& a, int threads, bool e4m3, cudaStream_t stream) {
  if (e4m3)
    launch_pdl(add_rmsnorm_kernel<kChunks, kVec, kRes, true>, a.num_tokens, threads, stream, a);
  else
    launch_pdl(add_rmsnorm_kernel<kChunks, kVec, kRes, false>, a.num_tokens, threads, stream, a);
}

template <int kChunks, bool kVec>
static void launch_norm_res(const NormArgs& a, int threads, int res, bool e4m3, cudaStream_t stream) {
  if (res == 0)
    launch_norm_out<kChunks, kVec, 0>(a, threads, e4m3, stream);
  else if (res == 1)
    launch_norm_out<kChunks, kVec, 1>(a, threads, e4m3, stream);
  else
    launch_norm_out<kChunks, kVec, 2>(a, threads, e4m3, stream);
}

}  // namespace mla_nq

namespace mla {

// residual_kind: 0 none, 1 bf16, 2 fp32.  Arguments are checked by the caller.
cudaError_t launch_add_rmsnorm(const void* x, int64_t x_stride, const void* res_in, void* res_out, int residual_kind,
                               int64_t res_stride, const void* weight, int num_tokens, int dim, float eps, void* y,
                               int64_t y_stride, bool e4m3, float* y_scales, int64_t scale_stride,
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
  const int items = (dim + 7) / 8;
  const int chunks = items <= 1024 ? 1 : items <= 2048 ? 2 : 4;
  const int threads = ((items + chunks - 1) / chunks + 31) / 32 * 32;
  if (chunks == 1)
    vec ? launch_norm_res<1, true>(a, threads, residual_kind, e4m3, stream)
        : launch_norm_res<1, false>(a, threads, residual_kind, e4m3, stream);
  else if (chunks == 2)
    vec ? launch_norm_res<2, true>(a, threads, residual_kind, e4m3, stream)
        : launch_norm_res<2, false>(a, threads, residual_kind, e4m3, stream);
  else
    vec ? launch_norm_res<4, true>(a, threads, residual_kind, e4m3, stream)
        : launch_norm_res<4, false>(a, threads, residual_kind, e4m3, stream);
  return cudaGetLastError();
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
  a.dim = dim;
  a.items_per_row = (dim + 127) / 128 * 16;
  a.items = (int64_t)num_tokens * a.items_per_row;
  const bool vec = dim % 8 == 0 && x_stride % 8 == 0 && y_stride % 8 == 0 && multiple(x, 16) && multiple(y, e4m3 ? 8 : 16);
  const unsigned blocks = (unsigned)((a.items + kActThreads - 1) / kActThreads);
  if (silu_mul && e4m3)
    vec ? launch_pdl(act_quantize_kernel<true, true, true>, blocks, kActThreads, stream, a)
        : launch_pdl(act_quantize_kernel<false, true, true>, blocks, kActThreads, stream, a);
  else if (silu_mul)
    vec ? launch_pdl(act_quantize_kernel<true, true, false>, blocks, kActThreads, stream, a)
        : launch_pdl(act_quantize_kernel<false, true, false>, blocks, kActThreads, stream, a);
  else
    vec ? launch_pdl(act_quantize_kernel<true, false, true>, blocks, kActThreads, stream, a)
        : launch_pdl(act_quantize_kernel<false, false, true>, blocks, kActThreads, stream, a);
  return cudaGetLastError();
}

}  // namespace mla
