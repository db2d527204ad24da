// out[m][n] = sum over blocks b of 128 of xs[m][b] ws[n / 128][b] sum_{k in b} x[m][k] w[n][k]
//
// x and w hold e4m3 codes.  A block's products are one step of
// v_mfma_f32_16x16x128_f8f6f4, whose result is scaled in fp32 and added to the
// running sums.
#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

namespace {
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma128(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
__device__ const uint4 kZeros = {0, 0, 0, 0};

// A lane's 32 codes of row `row` in block b: pieces g4 and g4 + 4 of 16 (the same
// for both operands, so their order in the block does not matter); 0 from k on
__device__ __forceinline__ i32x8 codes_of(const uint8_t* row, int64_t b, int g4, int64_t k) {
  const int64_t c0 = b * 128 + g4 * 16, c1 = c0 + 64;
  const i32x4 lo = *reinterpret_cast<const i32x4*>(c0 < k ? row + c0 : reinterpret_cast<const uint8_t*>(&kZeros));
  const i32x4 hi = *reinterpret_cast<const i32x4*>(c1 < k ? row + c1 : reinterpret_cast<const uint8_t*>(&kZeros));
  return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}
}  // namespace

// A wave takes 16 rows of w and 16 of x.
__global__ void __launch_bounds__(256) k_matmul_q8_simple(const MatmulArgs a) {
  const int lane = threadIdx.x & 63, g4 = lane >> 4, c16 = lane & 15;
  const int64_t tiles_n = (a.n + 15) / 16;
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t n0 = tile % tiles_n * 16, m0 = tile / tiles_n * 16;
  if (m0 >= a.m) return;
  const int64_t across = (a.k + 127) / 128;
  const int64_t m = min(m0 + c16, a.m - 1);
  const uint8_t* const w = a.w + min(n0 + c16, a.n - 1) * a.w_st;
  const uint8_t* const x = a.x + m * a.x_st;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int64_t b = 0; b < across; ++b) {
    const f32x4 p = mfma128(codes_of(w, b, g4, a.k), codes_of(x, b, g4, a.k), f32x4{0.f, 0.f, 0.f, 0.f});
    const float s = a.xs[m * across + b] * a.ws[n0 / 128 * across + b];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(p[i], s, sum[i]);
  }
  // sum[i]: column n0 + 4 g4 + i of row m0 + c16
  if (m0 + c16 >= a.m) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + 4 * g4 + i < a.n) a.out[m * a.o_st + n0 + 4 * g4 + i] = (uint16_t)(pk_bf16(sum[i], 0.f) & 0xFFFFu);
}

bool matmul_q8_fits(int64_t m, int64_t n, int64_t k) { return ((m + 15) / 16) * ((n + 15) / 16) < ((int64_t)1 << 25); }

size_t matmul_q8_workspace_bytes(int64_t m, int64_t n, int64_t k) { return 0; }

hipError_t launch_matmul_q8(const MatmulArgs& a, void* work, hipStream_t st) {
  const int64_t tiles = ((a.m + 15) / 16) * ((a.n + 15) / 16);
  hipLaunchKernelGGL(k_matmul_q8_simple, dim3((unsigned)((tiles + 3) / 4)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace misa
