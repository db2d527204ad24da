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
// 16 bytes a lane from a buffer into LDS (dst: the wave's 1 KB, lane order)
typedef __attribute__((address_space(3))) void* lds_void;
__device__ __forceinline__ void stage16(__amdgpu_buffer_rsrc_t r, unsigned char* dst, uint32_t off, uint32_t block) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void)dst, 16, off, block * 128, 0, 0);
}

// What a launch adds to the arguments
struct Plan {
  int tiles_n, tiles_m;   // output tiles
  int splits, per;        // parts of the blocks, and blocks of a part
  float* part;            // splits > 1: the parts' sums [split][m][n]
};
}  // namespace

// A workgroup of WN x WM waves takes (16 FN WN) rows of w by (16 FM WM) rows of x, a
// wave 16 FN by 16 FM of them.  A block's codes are staged in LDS for all waves, the
// next block's while this one is multiplied; row r's piece c of 16 bytes lies at c ^ (r
// & 7), so eight rows' reads of a piece meet no bank twice.
template <int WN, int WM, int FN, int FM>
__global__ void __launch_bounds__(WN * WM * kWave, WN * WM == 8 ? 2 : 2) k_matmul_tile(const MatmulArgs a, const Plan pl) {
  constexpr int NW = WN * WM, BN = 16 * FN * WN, BM = 16 * FM * WM;
  constexpr int LN = BN / 8 / NW, LM = BM / 8 / NW;   // loads of a wave: 8 rows each
  __shared__ __attribute__((aligned(16))) unsigned char s_w0[BN * 128], s_w1[BN * 128], s_x0[BM * 128], s_x1[BM * 128];
  const int lane = threadIdx.x & 63, g4 = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN;

  // tiles of an XCD's workgroups side by side: 8 rows of tiles at a time, down first
  int id = (int)xcd_remap(blockIdx.x, (int64_t)pl.tiles_n * pl.tiles_m * pl.splits);
  const int split = id % pl.splits;
  id /= pl.splits;
  constexpr int kDeep = 8;
  const int band = id / (kDeep * pl.tiles_n), deep = min(kDeep, pl.tiles_m - band * kDeep);
  id -= band * kDeep * pl.tiles_n;
  const int64_t m0 = (int64_t)(band * kDeep + id % deep) * BM, n0 = (int64_t)(id / deep) * BN;
  const int across = (int)((a.k + 127) / 128);
  const int b0 = split * pl.per, b1 = min(across, b0 + pl.per);
  const int kend = min((int)a.k, b1 * 128);

  const int rows_n = (int)min((int64_t)BN, a.n - n0), rows_m = (int)min((int64_t)BM, a.m - m0);
  const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(a.w + n0 * a.w_st, (uint32_t)((rows_n - 1) * a.w_st + a.k));
  const __amdgpu_buffer_rsrc_t rx = uniform_rsrc(a.x + m0 * a.x_st, (uint32_t)((rows_m - 1) * a.x_st + a.k));
  // rows past the last repeat it; their results are not written
  uint32_t ow[LN], ox[LM];
  const int piece = (lane & 7) ^ (lane >> 3);   // (loads begin at multiples of 8 rows)
#pragma unroll
  for (int u = 0; u < LN; ++u) ow[u] = (uint32_t)min((u * NW + wave) * 8 + (lane >> 3), rows_n - 1) * (uint32_t)a.w_st + piece * 16;
#pragma unroll
  for (int u = 0; u < LM; ++u) ox[u] = (uint32_t)min((u * NW + wave) * 8 + (lane >> 3), rows_m - 1) * (uint32_t)a.x_st + piece * 16;
  const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(a.xs + m0 * across, (uint32_t)(rows_m * across) * 4u);
  uint32_t os[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) os[j] = (uint32_t)(min((wm * FM + j) * 16 + c16, rows_m - 1) * across) * 4u;
  const __amdgpu_buffer_rsrc_t rt = uniform_rsrc(a.ws + min(n0 + wn * FN * 16, a.n - 1) / 128 * across, (uint32_t)across * 4u);

  float s_next[FM], ws_next;
  auto issue = [&](int b, unsigned char* dw, unsigned char* dx) __attribute__((always_inline)) {
    // from kend on there are no codes: past the buffer's end, which reads as 0
    const uint32_t gone = b * 128 + piece * 16 >= kend ? 0x80000000u : 0u;
#pragma unroll
    for (int u = 0; u < LN; ++u) stage16(rw, dw + (u * NW + wave) * 1024, ow[u] | gone, b);
#pragma unroll
    for (int u = 0; u < LM; ++u) stage16(rx, dx + (u * NW + wave) * 1024, ox[u] | gone, b);
  };
  auto scales = [&](int b) __attribute__((always_inline)) {
    const uint32_t gone = b < b1 ? 0u : 0x80000000u;   // (0, so that nothing is added)
#pragma unroll
    for (int j = 0; j < FM; ++j) s_next[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, os[j] | gone, b * 4, 0));
    ws_next = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rt, gone, b * 4, 0));
  };

  f32x4 sum[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) sum[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // pieces g4 and g4 + 4 of row c16
  const int lo = c16 * 128 + ((g4 ^ (c16 & 7)) << 4);
  auto frag = [&](const unsigned char* s) __attribute__((always_inline)) {
    const i32x4 x = *reinterpret_cast<const i32x4*>(s + lo), y = *reinterpret_cast<const i32x4*>(s + (lo ^ 64));
    return i32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  };
  auto step = [&](int b, const unsigned char* cw, const unsigned char* cx, unsigned char* nw, unsigned char* nx) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();   // block b is in LDS, and nobody reads the other buffer any more
    float s[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) s[j] = s_next[j] * ws_next;
    issue(b + 1, nw, nx);
    scales(b + 1);
    i32x8 fx[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) fx[j] = frag(cx + (wm * FM + j) * 2048);
    // A row of products while the row before it is scaled and added
    i32x8 fw = frag(cw + wn * FN * 2048);
    f32x4 p[2][FM];
#pragma unroll
    for (int i = 0; i <= FN; ++i) {
      i32x8 next = fw;
      if (i + 1 < FN) next = frag(cw + (wn * FN + i + 1) * 2048);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        if (i < FN) p[i & 1][j] = mfma128(fw, fx[j], f32x4{0.f, 0.f, 0.f, 0.f});
        if (i > 0)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[i - 1][j][e] = __builtin_fmaf(p[(i - 1) & 1][j][e], s[j], sum[i - 1][j][e]);
      }
      __builtin_amdgcn_sched_barrier(0);
      fw = next;
    }
  };
  issue(b0, s_w0, s_x0);
  scales(b0);
  for (int b = b0; b < b1; b += 2) {   // (an odd last one is followed by a block of nothing)
    step(b, s_w0, s_x0, s_w1, s_x1);
    step(b + 1, s_w1, s_x1, s_w0, s_x0);
  }
  __builtin_amdgcn_s_waitcnt(0);   // no load into LDS outlives the workgroup

  // sum[i][j][e]: column 16 i + 4 g4 + e of row 16 j + c16 of the wave's part
  const bool wide = ((a.o_st | (int64_t)((uintptr_t)a.out >> 1)) & 3) == 0;
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int64_t m = m0 + (wm * FM + j) * 16 + c16;
    if (m >= a.m) continue;
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const int64_t n = n0 + (wn * FN + i) * 16 + 4 * g4;
      if (n >= a.n) continue;
      const f32x4 v = sum[i][j];
      if (pl.splits > 1) {
        float* const dst = pl.part + ((int64_t)split * a.m + m) * a.n + n;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.n) dst[e] = v[e];
        continue;
      }
      uint16_t* const dst = a.out + m * a.o_st + n;
      const uint2 y = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
      if (wide && n + 4 <= a.n) {
        *reinterpret_cast<uint2*>(dst) = y;
      } else {
        dst[0] = (uint16_t)(y.x & 0xFFFFu);
        if (n + 1 < a.n) dst[1] = (uint16_t)(y.x >> 16);
        if (n + 2 < a.n) dst[2] = (uint16_t)(y.y & 0xFFFFu);
        if (n + 3 < a.n) dst[3] = (uint16_t)(y.y >> 16);
      }
    }
  }
}

namespace {
template <int WN, int WM, int FN, int FM>
hipError_t launch_tile(const MatmulArgs& a, void* work, hipStream_t st) {
  constexpr int BN = 16 * FN * WN, BM = 16 * FM * WM;
  const int tn = (int)((a.n + BN - 1) / BN), tm = (int)((a.m + BM - 1) / BM);
  const Plan pl{tn, tm, 1, (int)((a.k + 127) / 128), nullptr};
  hipLaunchKernelGGL((k_matmul_tile<WN, WM, FN, FM>), dim3((unsigned)(tn * tm)), dim3(WN * WM * kWave), 0, st, a, pl);
  return hipGetLastError();
}
}  // namespace

bool matmul_q8_fits(int64_t m, int64_t n, int64_t k) { return ((m + 127) / 128) * ((n + 127) / 128) < ((int64_t)1 << 23); }

size_t matmul_q8_workspace_bytes(int64_t m, int64_t n, int64_t k) { return 0; }

hipError_t launch_matmul_q8(const MatmulArgs& a, void* work, hipStream_t st) {
  if (a.m * a.n >= (int64_t)256 * 256 * 200) return launch_tile<2, 4, 8, 4>(a, work, st);
  return launch_tile<2, 2, 4, 4>(a, work, st);
}

}  // namespace misa
