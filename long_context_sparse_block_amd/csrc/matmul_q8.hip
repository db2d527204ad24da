// out[m][n] = sum over blocks b of 128 of xs[m][b] ws[n / 128][b] sum_{k in b} x[m][k] w[n][k]
//
// x and w hold e4m3 codes.  A block's products are formed by the f8f6f4 matrix
// instructions (the only ones at the full e4m3 rate), each block's sum from 0; it is
// scaled in fp32 and added to the running sums, in the blocks' order (k_matmul_rows:
// eight runs of blocks, then joined), and the result is rounded to bf16 once.  The
// matrix unit sums eight neighbouring products at a time, each cut at 2^-13 of the
// largest (measured; the eights are added up without further loss): with codes of 4 bits
// and a result of 8 that costs nothing seen, the relative error of the results here is
// 0.0017 in all, bf16's own rounding.  w is the instructions' first operand, so that
// a lane's results are one row of x, whose scale is one factor a lane.
//
// Measured: 8192 x 8192 x 4096 272-282 us by card (1952 to 2018 TFLOP/s; the library's
// product of the same codes with one scale for all 211-227 us), 8192 x 4096 x 8192 258 us
// (2129); the clock falls to 1.75-1.9 GHz there, MFMA is busy 0.50-0.56 of the time, the
// vector unit 0.36-0.45.  515 x 4099 x 1504 12.5-14 us, 64 x 8192 x 2048 7.4-8.4 us, 1 x 8192 x
// 4096 7.1-7.9 us (33.6 MB, 4.3 to 4.7 TB/s).
// Tried on the large tiles and not kept: a workgroup that goes on to the next tile with
// its first block on the way (286 us; the results leave in smaller pieces, 18
// registers are spilled), a second barrier in the middle of a block to ask for the
// one after the next earlier (281), loads spread over all tiles of a block (280), 4 or 16
// tiles deep for an XCD instead of 8 (the same), raised wave priority around the
// products (295 against 288 on that card).
#include <algorithm>

#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

namespace {
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x4 mfma128(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma64(i32x8 a, i32x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
// 16 bytes a lane from a buffer into LDS (dst: the wave's 1 KB, lane order)
typedef __attribute__((address_space(3))) void* lds_void;
__device__ __forceinline__ void stage16(__amdgpu_buffer_rsrc_t r, unsigned char* dst, uint32_t off, uint32_t block) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void)dst, 16, off, block * 128, 0, 0);
}

constexpr int kValu = 0x2, kMfma = 0x8, kDsRead = 0x100;   // instruction classes of sched_group_barrier

// What a launch adds to the arguments
struct Plan {
  int tiles_n, tiles_m;   // output tiles
  int splits, per;        // parts of the blocks, and blocks of a part
  float* part;            // splits > 1: the parts' sums [split][ld / 4][m][4], so that a store's lanes fill lines
  int64_t ld;             // n, rounded up to 4
};
}  // namespace

// The same unknown to the compiler, which would otherwise wait for all loads into
// LDS before any read of the array that they fill.  Who reads waits: landed().
// (dst: offset in LDS, by way of m0, which the compiler writes; it does not count the wait state that a load into LDS
// takes behind that.  No vector register is written.)
template <int BYTES>
__device__ __forceinline__ void stage_far(__amdgpu_buffer_rsrc_t r, uint32_t dst, uint32_t off, uint32_t add) {
#ifdef __HIP_DEVICE_COMPILE__
  if constexpr (BYTES == 16)
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"{m0}"(dst), "v"(off), "s"(r), "s"(add) : "memory");
  else
    asm volatile("s_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"{m0}"(dst), "v"(off), "s"(r), "s"(add) : "memory");
#endif
}
// All of the workgroup's loads but each wave's last N have landed in LDS, and its reads are done
template <int N>
__device__ __forceinline__ void landed() {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
#endif
}

// A workgroup of WN x WM waves takes (32 FN WN) rows of w by (32 FM WM) rows of x, a
// wave 32 FN by 32 FM of them.  S blocks' codes and scales are in LDS or on their way
// there; row r's piece c of 16 bytes lies at c ^ (r / 2 & 7): a read of a piece takes
// 16 rows at a time, and two rows fill all banks.
//
// A block of a 32 x 32 tile is two matrix instructions of 64 cycles, between which
// the tile before is scaled and added: 16 vector instructions, where such an
// instruction leaves room for 12 beside it.  (Of 16 x 16 x 128 every second cycle of
// the vector unit is the matrix unit's own, 4 fit beside one, and its tile needs 4.)
// The last row of a block's tiles is multiplied behind the barrier, while the
// next block's first operands are read.  Loads go out behind that, with more than
// two blocks a few to a tile: a wave that asks for more than the CU takes in (64 bytes
// a cycle) stands still, and its products with it.
template <int WN, int WM, int FN, int FM, int S>
__global__ void __launch_bounds__(WN * WM * kWave, WN * WM / 4) k_matmul_tile(const MatmulArgs a, const Plan pl) {
  constexpr int NW = WN * WM, BN = 32 * FN * WN, BM = 32 * FM * WM;
  constexpr int LN = BN / 8 / NW, LM = BM / 8 / NW;   // loads of a wave: 8 rows each
  constexpr int kOps = LN + LM + 1;                   // and one of scales
  constexpr int kEarly = S == 2 ? kOps : (kOps + FN - 1) / FN;   // loads of a block in the last row of tiles
  constexpr int kTiles = FN > 1 ? (FN - 1) * FM : 1;                // tiles that share the others
  constexpr int kX = BN * 128, kXs = kX + BM * 128, kWs = kXs + BM * 4, kStage = kWs + 256;
  static_assert(NW > BM / 64 && S * kStage <= 160 * 1024, "a wave for w's scales; the LDS");
  __shared__ __attribute__((aligned(16))) unsigned char s_mem[S * kStage];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void)s_mem;
  const int lane = threadIdx.x & 63, h = lane >> 5, c32 = lane & 31;
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
  // Eight rows' buffer, as far as there are rows: what lies behind reads as 0
  auto eight = [&](const uint8_t* base, int64_t st, int row, int rows) __attribute__((always_inline)) {
    const int in = min(8, rows - row);
    return uniform_rsrc(base + (in > 0 ? row * st : 0), in > 0 ? (uint32_t)((in - 1) * st + a.k) : 0u);
  };
  __amdgpu_buffer_rsrc_t rw[LN], rx[LM];
#pragma unroll
  for (int u = 0; u < LN; ++u) rw[u] = eight(a.w + n0 * a.w_st, a.w_st, (u * NW + wave) * 8, rows_n);
#pragma unroll
  for (int u = 0; u < LM; ++u) rx[u] = eight(a.x + m0 * a.x_st, a.x_st, (u * NW + wave) * 8, rows_m);
  const int piece = (lane & 7) ^ (lane >> 4) ^ ((wave & 1) << 2);   // (a load's 8 rows begin at 8 (u NW + wave))
  const uint32_t ow = (uint32_t)(lane >> 3) * (uint32_t)a.w_st + piece * 16;
  const uint32_t ox = (uint32_t)(lane >> 3) * (uint32_t)a.x_st + piece * 16;
  // scales: a wave loads 64 rows of x, or (the last ones, all the same) w's rows of blocks
  const bool of_x = wave < BM / 64;
  const int srow = of_x ? wave * 64 : 0;
  const int srows = of_x ? max(0, min(64, rows_m - srow)) : (rows_n + 127) / 128;
  const __amdgpu_buffer_rsrc_t rs =
      uniform_rsrc(of_x ? a.xs + (srows > 0 ? (m0 + srow) * across : 0) : a.ws + n0 / 128 * across, (uint32_t)(srows * across) * 4u);
  const uint32_t os = (uint32_t)(lane * across) * 4u, sdst = of_x ? kXs + wave * 256 : kWs;

  // loads from .. to - 1 of the wave's kOps of block b: x, the scales, w
  auto issue = [&](int b, int stage, int from, int to) __attribute__((always_inline)) {
    const uint32_t base = lds0 + stage * kStage;
    // from kend on there are no codes: past the buffer's end too
    const uint32_t gone = b * 128 + piece * 16 >= kend ? 0x80000000u : 0u;
#pragma unroll
    for (int u = 0; u < kOps; ++u) {
      if (u < from || u >= to) continue;
      if (u < LM) stage_far<16>(rx[u < LM ? u : 0], base + kX + (u * NW + wave) * 1024, ox | gone, b * 128);
      else if (u == LM) stage_far<4>(rs, base + sdst, b < b1 ? os : 0x80000000u, b * 4);   // (0 there, so that nothing is added)
      else stage_far<16>(rw[u > LM ? u - LM - 1 : 0], base + ((u - LM - 1) * NW + wave) * 1024, ow | gone, b * 128);
    }
  };

  f32x16 sum[FN][FM], p;
#pragma unroll
  for (int e = 0; e < 16; ++e) p[e] = 0.f;
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) sum[i][j] = p;
  // A lane's codes of row c32: pieces h, 2 + h, 4 + h, 6 + h
  struct Frag {
    i32x8 k[2];
  };
  const int at = c32 * 128 + ((h ^ ((c32 >> 1) & 7)) << 4), at_w = at + wn * FN * 4096, at_x = at + wm * FM * 4096 + kX;
  auto frag = [&](const unsigned char* from, int lane_at) __attribute__((always_inline)) {
    i32x4 x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = *reinterpret_cast<const i32x4*>(from + (lane_at ^ (q << 5)));
    return Frag{{i32x8{x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]},
                 i32x8{x[2][0], x[2][1], x[2][2], x[2][3], x[3][0], x[3][1], x[3][2], x[3][3]}}};
  };
  const int at_s = kXs + (wm * FM * 32 + c32) * 4, at_t = kWs + (wn * FN * 32 / 128) * 4;
  float s_old, s[FM];   // of the tile before the block's first, of the block
  auto scales = [&](const unsigned char* from) __attribute__((always_inline)) {
    const float w = *reinterpret_cast<const float*>(from + at_t);
#pragma unroll
    for (int j = 0; j < FM; ++j) s[j] = *reinterpret_cast<const float*>(from + at_s + j * 128) * w;
  };
  Frag fx[FM], fw;

#pragma unroll
  for (int b = 0; b < S - 1; ++b) issue(b0 + b, b, 0, kOps);
  issue(b0 + S - 1, S - 1, 0, kEarly);
  landed<(S - 2) * kOps + kEarly>();
#pragma unroll
  for (int j = 0; j < FM; ++j) fx[j] = frag(s_mem + j * 4096, at_x);
  fw = frag(s_mem, at_w);
#pragma unroll
  for (int j = 0; j < FM; ++j) s[j] = 0.f;
  int stage = 0;
  for (int b = b0; b < b1; ++b) {
    const int after = stage + 1 < S ? stage + 1 : 0;
    const unsigned char* const cur = s_mem + stage * kStage;
    const unsigned char* const nxt = s_mem + after * kStage;
    s_old = s[FM - 1];
    scales(cur);
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      if (i == FN - 1) landed<(S - 2) * kOps>();   // block b + 1 is in LDS, and nobody reads block b there any more
      const Frag next = i + 1 < FN ? frag(cur + (i + 1) * 4096, at_w) : frag(nxt, at_w);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const int before = i * FM + j - 1;   // the tile whose products are scaled and added
        f32x16& to = before < 0 ? sum[FN - 1][FM - 1] : sum[before / FM][before % FM];
        const float sc = before < 0 ? s_old : s[before % FM];
        f32x16 y;
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = 0.f;
        y = mfma64(fw.k[0], fx[j].k[0], y);
        y = mfma64(fw.k[1], fx[j].k[1], y);
#pragma unroll
        for (int e = 0; e < 16; ++e) to[e] = __builtin_fmaf(p[e], sc, to[e]);
        p = y;
        if (i == FN - 1) {
          fx[j] = frag(nxt + j * 4096, at_x);
          issue(b + S, stage, j * kEarly / FM, (j + 1) * kEarly / FM);   // behind the reads: a load waits for those before it
        } else {
          constexpr int late = kOps - kEarly;
          const int n = i * FM + j;
          issue(b + S - 1, stage > 0 ? stage - 1 : S - 1, kEarly + n * late / kTiles, kEarly + (n + 1) * late / kTiles);
        }
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kValu, 8, 0);
        __builtin_amdgcn_sched_group_barrier(kDsRead, 4, 0);
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kValu, 8, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      fw = next;
    }
    stage = after;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) sum[FN - 1][FM - 1][e] = __builtin_fmaf(p[e], s[FM - 1], sum[FN - 1][FM - 1][e]);
  landed<0>();   // no load into LDS outlives the workgroup, and nothing is read there any more

  // sum[i][j][4 q + e]: column 32 i + 8 q + 4 h + e of row 32 j + c32 of the wave's part
  const int64_t mw = m0 + wm * FM * 32, nw = n0 + wn * FN * 32;
  if (pl.splits > 1) {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int64_t m = mw + j * 32 + c32;
      float* const dst = pl.part + (int64_t)split * a.m * pl.ld + nw * a.m + m * 4;
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (m < a.m && nw + i * 32 + 8 * q + 4 * h < a.n)
            *reinterpret_cast<f32x4*>(dst + (i * 32 + 8 * q + 4 * h) * a.m) =
                f32x4{sum[i][j][4 * q], sum[i][j][4 * q + 1], sum[i][j][4 * q + 2], sum[i][j][4 * q + 3]};
    }
    return;
  }
  // Through LDS, so that rows are written 16 bytes a lane and side by side: from
  // the lanes that hold them they go out in pieces of 16 bytes, and took as long as a
  // quarter of the products (8192 x 8192 x 4096).  Row r's piece c lies at c ^ r.
  constexpr int P = FN * 4, RP = kWave / P;   // pieces of a row, rows of a store
  static_assert(NW * FM * 32 * P * 16 <= S * kStage, "the waves' rows fit");
  unsigned char* const mine = s_mem + wave * (FM * 32 * P * 16);
#pragma unroll
  for (int j = 0; j < FM; ++j)
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint2*>(mine + (j * 32 + c32) * P * 16 + (((i * 4 + q) ^ (c32 & (P - 1))) << 4) + h * 8) =
            make_uint2(pk_bf16(sum[i][j][4 * q], sum[i][j][4 * q + 1]), pk_bf16(sum[i][j][4 * q + 2], sum[i][j][4 * q + 3]));
  if (((a.o_st | (int64_t)((uintptr_t)a.out >> 1)) & 7) == 0) {
    const int row = lane / P, col = lane % P;
    const int64_t n = nw + col * 8;
#pragma unroll
    for (int r = 0; r < FM * 32; r += RP) {
      const uint4 y = *reinterpret_cast<const uint4*>(mine + (r + row) * P * 16 + ((col ^ ((r + row) & (P - 1))) << 4));
      const int64_t m = mw + r + row;
      if (m >= a.m || n >= a.n) continue;
      uint16_t* const dst = a.out + m * a.o_st + n;
      if (n + 8 <= a.n) {
        *reinterpret_cast<uint4*>(dst) = y;
      } else {
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < a.n) dst[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
      }
    }
    return;
  }
  // rows that begin anywhere: a column a lane (515 x 4099 x 1504: 13.2-13.7 us, with 8 a lane 15.0, with
  // aligned pieces of 16 bytes and the columns beside them apart 23)
  constexpr int W = FN * 32 < kWave ? FN * 32 : kWave;   // columns of a store
  const int row = lane / W, col = lane % W;
#pragma unroll 4
  for (int i = 0; i < FM * 32 * FN * 32 / kWave; ++i) {
    const int r = i / (FN * 32 / W) * (kWave / W) + row, c = i % (FN * 32 / W) * W + col;
    const uint16_t y = *reinterpret_cast<const uint16_t*>(mine + r * P * 16 + (((c / 8) ^ (r & (P - 1))) << 4) + (c & 7) * 2);
    if (mw + r < a.m && nw + c < a.n) a.out[(mw + r) * a.o_st + nw + c] = y;
  }
}

// Few rows of x (at most 16 MT; not of the longest): bound by the reading of w.  A workgroup takes 16 NT
// rows of w, each of its 8 waves an eighth of their blocks; their sums join in LDS, always
// in the same order.  w's codes go straight to the registers that the
// products read them from, x's through the wave's own LDS (side by side there, a row's
// lanes are apart in the registers' order, which loads at a third of the rate), both a
// block ahead, so that no barrier stands between a wave and its loads.
template <int NT, int MT>
__global__ void __launch_bounds__(8 * kWave, 2) k_matmul_rows(const MatmulArgs a) {
  constexpr int kXBytes = MT * 2048, kWaves = 8;
  constexpr int kJoin = kWaves * NT * MT * kWave * 16;
  constexpr int kBuf = kWaves * kXBytes;
  __shared__ __attribute__((aligned(16))) unsigned char s_x0[kJoin > kBuf ? kJoin : kBuf], s_x1[kBuf];
  const int lane = threadIdx.x & 63, g4 = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NT;
  const int across = (int)((a.k + 127) / 128);
  const int rows_m = (int)a.m, rows_n = (int)min((int64_t)16 * NT, a.n - n0);

  const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(a.w + n0 * a.w_st, (uint32_t)((rows_n - 1) * a.w_st + a.k));
  const __amdgpu_buffer_rsrc_t rx = uniform_rsrc(a.x, (uint32_t)((rows_m - 1) * a.x_st + a.k));
  const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(a.xs, (uint32_t)(rows_m * across) * 4u);
  const __amdgpu_buffer_rsrc_t rt = uniform_rsrc(a.ws + n0 / 128 * across, (uint32_t)across * 4u);
  // rows past the last repeat it; their results are not written
  const int piece = (lane & 7) ^ (lane >> 3);
  uint32_t ow[NT], ox[2 * MT], os[MT];
#pragma unroll
  for (int i = 0; i < NT; ++i) ow[i] = (uint32_t)min(i * 16 + c16, rows_n - 1) * (uint32_t)a.w_st + g4 * 16;
#pragma unroll
  for (int u = 0; u < 2 * MT; ++u) ox[u] = (uint32_t)min(u * 8 + (lane >> 3), rows_m - 1) * (uint32_t)a.x_st + piece * 16;
#pragma unroll
  for (int j = 0; j < MT; ++j) os[j] = (uint32_t)(min(j * 16 + c16, rows_m - 1) * across) * 4u;

  // the wave's blocks
  const int per = (across + kWaves - 1) / kWaves, b0 = min(wave * per, across), b1 = min(b0 + per, across);
  const int k = min((int)a.k, b1 * 128);
  struct Codes {
    i32x4 w[NT][2];
  };
  // scales of four blocks: a lane's of one block are as many lines apart as of four.  Past the last block they are the
  // next row's, or, behind the last row's, 0 without a read: the unit's bounds check takes in the scalar offset (the
  // builtin's documentation leaves it out) and goes by single dwords, as measured on buffers that end before their
  // memory does, with offsets before and past the end, to registers and to LDS.
  struct Scales {
    f32x4 x[MT], w;
  };
  auto four = [&](int b, Scales& c) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < MT; ++j) c.x[j] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, os[j], b * 4, 0));
    c.w = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rt, 0, b * 4, 0));
  };
  auto issue = [&](int b, unsigned char* dst, Codes& c) __attribute__((always_inline)) {
    // behind the last column there are no codes: past the buffers' ends, which read as 0
    const uint32_t gone = b * 128 + piece * 16 >= k ? 0x80000000u : 0u;
#pragma unroll
    for (int u = 0; u < 2 * MT; ++u) stage16(rx, dst + u * 1024, ox[u] | gone, b);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        c.w[i][q] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  rw, (ow[i] + q * 64) | (b * 128 + q * 64 + g4 * 16 >= k ? 0x80000000u : 0u), b * 128, 0));
  };
  constexpr int kOps = 2 * MT + 2 * NT;   // loads of a block

  f32x4 sum[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) sum[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int at = c16 * 128 + ((g4 ^ (c16 & 7)) << 4);   // pieces g4 and g4 + 4 of row c16
  auto multiply = [&](int b, const unsigned char* x, const Codes& c, const Scales& sc, int e4) __attribute__((always_inline)) {
    const float ws = b < b1 ? sc.w[e4] : 0.f;   // (behind the wave's blocks the codes are 0, the scales another's)
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(x + j * 2048 + at), hi = *reinterpret_cast<const i32x4*>(x + j * 2048 + (at ^ 64));
      const i32x8 fx = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      const float s = b < b1 ? sc.x[j][e4] * ws : 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const i32x4 p0 = c.w[i][0], p1 = c.w[i][1];
        const f32x4 p = mfma128(i32x8{p0[0], p0[1], p0[2], p0[3], p1[0], p1[1], p1[2], p1[3]}, fx, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[i][j][e] = __builtin_fmaf(p[e], s, sum[i][j][e]);
      }
    }
  };
  unsigned char* const x0 = s_x0 + wave * kXBytes;
  unsigned char* const x1 = s_x1 + wave * kXBytes;
  Codes c0, c1;
  Scales sc, next;
  four(b0, sc);
  issue(b0, x0, c0);
  auto step = [&](int b, int e4, unsigned char* cur, Codes& c, unsigned char* nxt, Codes& n) __attribute__((always_inline)) {
    issue(b + 1, nxt, n);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(kOps));   // all but what has just been asked for
    __builtin_amdgcn_sched_barrier(0);
    multiply(b, cur, c, sc, e4);
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int b = b0; b < b1; b += 4) {   // (blocks past the last add nothing)
    four(b + 4, next);
    step(b, 0, x0, c0, x1, c1);
    step(b + 1, 1, x1, c1, x0, c0);
    if (b + 2 >= b1) break;
    step(b + 2, 2, x0, c0, x1, c1);
    step(b + 3, 3, x1, c1, x0, c0);
    sc = next;
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  // sum[i][j][e]: column 16 i + 4 g4 + e of row 16 j + c16
  f32x4* const join = reinterpret_cast<f32x4*>(s_x0);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) join[(wave * NT * MT + i * MT + j) * kWave + lane] = sum[i][j];
  __syncthreads();
  if (wave >= NT * MT) return;
  f32x4 v = join[wave * kWave + lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v += join[(w * NT * MT + wave) * kWave + lane];
  const int64_t m = wave % MT * 16 + c16, n = n0 + wave / MT * 16 + 4 * g4;
  if (m >= a.m || n >= a.n) return;
  uint16_t* const dst = a.out + m * a.o_st + n;
  const uint2 y = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
  if (n + 4 <= a.n && ((uintptr_t)dst & 7) == 0) {
    *reinterpret_cast<uint2*>(dst) = y;
  } else {
    const uint32_t w[2] = {y.x, y.y};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.n) dst[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
  }
}

// The sums of a tile launch's parts, four columns of a row a thread, eight rows side by side
__global__ void __launch_bounds__(256) k_matmul_join(const MatmulArgs a, const Plan pl) {
  const int64_t quads = pl.ld / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t rows = i / (quads * 8), at = i - rows * quads * 8, m = rows * 8 + at % 8, n = at / 8 * 4;
  if (m >= a.m) return;
  const float* const src = pl.part + n * a.m + m * 4;
  f32x4 v = *reinterpret_cast<const f32x4*>(src);
#pragma unroll 8
  for (int s = 1; s < pl.splits; ++s) v += *reinterpret_cast<const f32x4*>(src + (int64_t)s * a.m * pl.ld);
  uint16_t* const dst = a.out + m * a.o_st + n;
  const uint2 y = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
  if (n + 4 <= a.n && ((uintptr_t)dst & 7) == 0) {
    *reinterpret_cast<uint2*>(dst) = y;
  } else {
    const uint32_t w[2] = {y.x, y.y};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.n) dst[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
  }
}

namespace {
// How a product is made.  The times are of a block of 128 columns: alone on their
// CUs, tiles of 64 x 64 take 0.3 us, 128 x 64 0.38, 128 x 128 0.47 to 0.65 (by how many
// there are); two of 128 x 128 on a CU 1.25, one of 256 x 256 2.1; 4 to 8 us a round
// beside.  Tiles that the card holds all at once may take parts of the blocks side by
// side, as many as it holds; the parts are then written and read again (at 6 TB/s, and
// 2.5 us more).  Whole against in parts: 105 x 555 x 2464 10.3 and 8.1 us, 512 x 2048 x 7168
// (256 tiles of 64 x 64 against four parts of 128 x 128) 22.5 and 20.0, 1024 x 1024 x 8192 26.6
// and 22.5; 515 x 1003 x 3600 and what is shorter stays whole.  Few rows: 64 x 1024 x 16384 by
// k_matmul_rows 22.4, in parts of tiles 10.4, 64 x 128 x 8192 12.4 and 9.1, 64 x 128 x 4096 8.1 and 8.3.
// (Few rows' times here are those of up to some 4096 columns: of more, of long rows, a workgroup's reading of x and
// the card's of w come on top, 64 x 8192 x 8192 19.4-19.8 us for the 12.5 that are reckoned.)
enum Form { kRows, kTile64, kTile128x64, kTile128, kTwo128, kTile256 };
struct Choice {
  Form form;
  int splits, per;
};
Choice choose(int64_t m, int64_t n, int64_t k) {
  const int64_t across = (k + 127) / 128;
  if (m == 0) return Choice{kRows, 1, (int)across};   // nothing to make
  auto tiles = [&](int bn, int bm) { return ((n + bn - 1) / bn) * ((m + bm - 1) / bm); };
  const double two = (double)((tiles(128, 128) + 511) / 512) * (1.25 * (double)across + 5.0);
  const double large = (double)((tiles(256, 256) + 255) / 256) * (2.1 * (double)across + 8.0);
  Choice best{two < large ? kTwo128 : kTile256, 1, (int)across};
  double least = std::min(two, large);
  constexpr struct { Form form; int bn, bm; double block; } small[] = {
      {kTile64, 64, 64, 0.3}, {kTile128x64, 128, 64, 0.38}, {kTile128, 128, 128, 0.5}};
  bool fits = false;
  if (m <= 64) {   // (an eighth of the blocks one after another: where that is long, parts of tiles)
    const double alone = m <= 16 ? 2.45 : m <= 32 ? 2.9 : 3.65, block = m <= 16 ? 0.6 : m <= 32 ? 0.78 : 1.1;
    best = Choice{kRows, 1, (int)across};
    least = alone + block * (double)((across + 7) / 8);
    fits = true;
  }
  for (const auto& f : small) {
    const int64_t held = 256 / tiles(f.bn, f.bm);   // parts that the card holds
    for (int64_t s = 1; s <= held && (s == 1 || across >= 4 * s); ++s) {
      const int64_t per = (across + s - 1) / s;
      if (s > 1 && (across + per - 1) / per != s) continue;
      const double cost = f.block * (double)per + 4.5 + (s > 1 ? 2.5 + 8.0 * (double)(s * m * n) / 6e6 : 0.0);
      if (fits && cost >= 0.95 * least) continue;   // (of nearly equal ones the smaller form, and fewer parts)
      fits = true;
      least = cost;
      best = Choice{f.form, (int)s, (int)per};
    }
  }
  return best;
}

template <int WN, int WM, int FN, int FM, int S>
hipError_t launch_tile(const MatmulArgs& a, const Choice& c, void* work, hipStream_t st) {
  constexpr int BN = 32 * FN * WN, BM = 32 * FM * WM;
  const int tn = (int)((a.n + BN - 1) / BN), tm = (int)((a.m + BM - 1) / BM);
  const Plan pl{tn, tm, c.splits, c.per, static_cast<float*>(work), (a.n + 3) / 4 * 4};
  hipLaunchKernelGGL((k_matmul_tile<WN, WM, FN, FM, S>), dim3((unsigned)(tn * tm * c.splits)), dim3(WN * WM * kWave), 0, st, a, pl);
  if (c.splits > 1)
    hipLaunchKernelGGL(k_matmul_join, dim3((unsigned)(((a.m + 7) / 8 * 8 * pl.ld / 4 + 255) / 256)), dim3(256), 0, st, a, pl);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_rows(const MatmulArgs& a, hipStream_t st) {
  // 16 rows of w to a workgroup where 32 would leave CUs without one
  if (a.n <= 16 * 256)
    hipLaunchKernelGGL((k_matmul_rows<1, MT>), dim3((unsigned)((a.n + 15) / 16)), dim3(8 * kWave), 0, st, a);
  else
    hipLaunchKernelGGL((k_matmul_rows<2, MT>), dim3((unsigned)((a.n + 31) / 32)), dim3(8 * kWave), 0, st, a);
  return hipGetLastError();
}
}  // namespace

// (a grid of fewer than 2^23 workgroups)
bool matmul_q8_fits(int64_t m, int64_t n, int64_t k) { return ((m + 127) / 128) * ((n + 127) / 128) < ((int64_t)1 << 23); }

size_t matmul_q8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  const Choice c = choose(m, n, k);
  return c.splits > 1 ? (size_t)c.splits * (size_t)m * (size_t)((n + 3) / 4 * 4) * sizeof(float) : 0;
}

hipError_t launch_matmul_q8(const MatmulArgs& a, void* work, hipStream_t st) {
  const Choice c = choose(a.m, a.n, a.k);
  switch (c.form) {
    case kRows: return a.m <= 16 ? launch_rows<1>(a, st) : a.m <= 32 ? launch_rows<2>(a, st) : launch_rows<4>(a, st);
    case kTile64: return launch_tile<2, 2, 1, 1, 3>(a, c, work, st);
    case kTile128x64: return launch_tile<2, 2, 2, 1, 3>(a, c, work, st);
    case kTile128: return launch_tile<2, 4, 2, 1, 3>(a, c, work, st);
    case kTwo128: return launch_tile<2, 2, 2, 2, 2>(a, c, work, st);
    default: return launch_tile<2, 4, 4, 2, 2>(a, c, work, st);
  }
}

}  // namespace misa
