// e4m3 codes of a matrix, with a scale for each block of 1 x 128 (activations) or
// 128 x 128 (weights): the operands of misa_matmul_q8.
//   scale = fp32(amax / 448), at least 2^-126; 1 for a block of zeros
//   code  = e4m3fn round-to-nearest-even of fp32(x / scale)
// with both divisions correctly rounded, so that codes are a fixed function of the
// input.  (At a scale below the smallest normal number the quotients would lose
// bits, or pass 448.)
//
// Bound by HBM, the quotients close behind (8192 x 4096 in bf16: 16.5-17.3 us, 101 MB,
// the vector unit busy 0.86 of it; with true divisions 19.9).  64 x 2048: 2.8 us,
// a launch's.
#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

namespace {
// 8 values of a row, as loaded
template <int DT> struct Eight {
  uint4 v;
  __device__ __forceinline__ void load(const void* p) { v = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    const uint32_t h = i & 1 ? w >> 16 : w & 0xFFFFu;
    if constexpr (DT == MISA_T_FP16) return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
    return bf16_bits_to_f32(h);
  }
};
template <> struct Eight<MISA_T_FP32> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = static_cast<const float4*>(p)[0];
    b = static_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ float at(int i) const {
    const float4 x = i < 4 ? a : b;
    return (i & 3) == 0 ? x.x : (i & 3) == 1 ? x.y : (i & 3) == 2 ? x.z : x.w;
  }
};

template <int DT>
__device__ __forceinline__ float amax8(const Eight<DT>& x) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = __builtin_fmaxf(a, __builtin_fabsf(x.at(i)));
  return a;
}
__device__ __forceinline__ float scale_of(float amax) {
  return amax > 0.f ? __builtin_fmaxf(__fdiv_rn(amax, 448.f), 0x1p-126f) : 1.f;
}
// fp32(x / s) by s's reciprocal r: the quotient of x r, corrected twice by what it
// leaves of x.  After the first it is one of the two floats about x / s, and from
// there, with r = fp32(1 / s) and an exact remainder, the second rounds x / s
// correctly (Markstein's theorem on division); 6 instructions where a division is
// 10, of 16 values to a lane.  The remainders are exact while s stays away from the
// ends of the range (quotients that round to code 0 aside).
__device__ __forceinline__ bool plain(float s) { return s >= 0x1p-80f && s <= 0x1p120f; }
__device__ __forceinline__ float quotient(float x, float s, float r) {
  float q = x * r;
  q = __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
  q = __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
  return __builtin_copysignf(q, x);   // (-0 / s)
}
template <int DT>
__device__ __forceinline__ uint2 codes8(const Eight<DT>& x, float s, float r, bool fast) {
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quotient(x.at(4 * h + i), s, r);
    if (!fast)
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = __fdiv_rn(x.at(4 * h + i), s);
    int v = 0;
    v = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], v, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], v, true);
    c[h] = (uint32_t)v;
  }
  return make_uint2(c[0], c[1]);
}
}  // namespace

// 8 lanes a block of 1 x 128, 16 values each (so that codes go out 16 bytes a lane)
template <int DT>
__global__ void __launch_bounds__(256) k_quant_rows(const char* __restrict__ x, int64_t x_bytes, int64_t rows, int64_t cols,
                                                    uint32_t across, uint8_t* __restrict__ codes, float* __restrict__ scale) {
  constexpr int E = DT == MISA_T_FP32 ? 4 : 2;
  const uint32_t block = blockIdx.x * 32 + threadIdx.x / 8, row = block / across;   // (fewer than 2^27 blocks)
  const int64_t r = row, c = (int64_t)(block - row * across) * 128 + (threadIdx.x & 7) * 16;
  const bool in = r < rows && c < cols;
  Eight<DT> v, w;
  v.zero();
  w.zero();
  if (in) {
    v.load(x + r * x_bytes + c * E);
    w.load(x + r * x_bytes + (c + 8) * E);
  }
  float amax = __builtin_fmaxf(amax8(v), amax8(w));
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o, 8));
  const float s = scale_of(amax);
  if (!in) return;
  const float recip = __fdiv_rn(1.f, s);
  const bool fast = plain(s);
  const uint2 a = codes8(v, s, recip, fast), b = codes8(w, s, recip, fast);
  *reinterpret_cast<uint4*>(codes + r * cols + c) = make_uint4(a.x, a.y, b.x, b.y);
  if ((threadIdx.x & 7) == 0) scale[block] = s;
}

// A workgroup a block of 128 x 128: thread t takes piece t % 16 of rows t / 16 + 16 i
template <int DT>
__global__ void __launch_bounds__(256) k_quant_squares(const char* __restrict__ x, int64_t x_bytes, int64_t rows, int64_t cols,
                                                       uint32_t across, uint8_t* __restrict__ codes,
                                                       float* __restrict__ scale) {
  constexpr int E = DT == MISA_T_FP32 ? 4 : 2;
  __shared__ float s_max[4];
  const int64_t r0 = (int64_t)(blockIdx.x / across) * 128 + threadIdx.x / 16;
  const int64_t c = (int64_t)(blockIdx.x % across) * 128 + (threadIdx.x & 15) * 8;
  Eight<DT> v[8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i].zero();
    if (r0 + 16 * i < rows && c < cols) v[i].load(x + (r0 + 16 * i) * x_bytes + c * E);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, amax8(v[i]));
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o));
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = amax;
  __syncthreads();
  const float s = scale_of(__builtin_fmaxf(__builtin_fmaxf(s_max[0], s_max[1]), __builtin_fmaxf(s_max[2], s_max[3])));
  const float recip = __fdiv_rn(1.f, s);
  const bool fast = plain(s);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < rows && c < cols)
      *reinterpret_cast<uint2*>(codes + (r0 + 16 * i) * cols + c) = codes8(v[i], s, recip, fast);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
}

template <int DT>
static hipError_t launch_type(const char* x, int64_t rows, int64_t cols, int64_t x_st, int block_rows, uint8_t* codes,
                              float* scale, hipStream_t st) {
  const int64_t x_bytes = x_st * (DT == MISA_T_FP32 ? 4 : 2), across = (cols + 127) / 128;
  if (block_rows == 1)
    hipLaunchKernelGGL(k_quant_rows<DT>, dim3((unsigned)((rows * across + 31) / 32)), dim3(256), 0, st, x, x_bytes, rows,
                       cols, (uint32_t)across, codes, scale);
  else
    hipLaunchKernelGGL(k_quant_squares<DT>, dim3((unsigned)((rows + 127) / 128 * across)), dim3(256), 0, st, x, x_bytes,
                       rows, cols, (uint32_t)across, codes, scale);
  return hipGetLastError();
}

hipError_t launch_quantize_blocks(const void* x, int dtype, int64_t rows, int64_t cols, int64_t x_st, int block_rows,
                                  uint8_t* codes, float* scale, hipStream_t st) {
  const char* p = static_cast<const char*>(x);
  if (dtype == MISA_T_BF16) return launch_type<MISA_T_BF16>(p, rows, cols, x_st, block_rows, codes, scale, st);
  if (dtype == MISA_T_FP16) return launch_type<MISA_T_FP16>(p, rows, cols, x_st, block_rows, codes, scale, st);
  return launch_type<MISA_T_FP32>(p, rows, cols, x_st, block_rows, codes, scale, st);
}

}  // namespace misa
