// What the attention kernels share (attn_tile.hip: many query rows against
// shared key tiles; attn_wave.hip: few query rows, each wave its own keys).
//
// Rows.  A kv head's query rows of a sequence are (new token, query head of
// the group): row r is token r / G, head r % G, G = n_heads / n_kv_heads.  A
// key tile then serves all G heads at once.  Over selected tokens the rows
// of a unit are one token's G heads.
//
// Both kernels form S^T = K Q^T, so a lane of the result holds one query row's
// scores (16 or 8 of a tile's keys): the softmax needs almost no lane
// exchange, the output's rescaling is one factor per lane, and the weights
// are already laid out as the second operand of O^T = V^T P^T, up to an order
// of the keys that V's reads follow.
//
// LDS tiles hold bf16 rows in 16-byte pieces, piece c of row r at position
// c ^ swizzle(r): K rows are then read 16 at a time, and V four rows at a time
// by gfx950's transposing read, without more lanes per bank than the read's
// size needs.
#pragma once

#include <math.h>

#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

constexpr float kLn2 = 0.6931471805599453f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_void;
typedef const __attribute__((address_space(1))) void* global_void;

// piece position of row r (D elements a row, D / 8 pieces)
template <int D>
__device__ __forceinline__ int swizzle(int r) {
  return D == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

// gfx950's transposing LDS read: lanes 4j .. 4j+3 of a 16-lane group name 4
// consecutive elements each of row j (j = 0..3); lane i of the group receives
// element i of the four rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 lds_read_tr(const unsigned char* p) {
  typedef __attribute__((address_space(3))) s16x4* ptr;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)p));
}

// 16 bytes a lane, global -> LDS (dst: the wave's 1 KB, lane order)
__device__ __forceinline__ void load_lds16(const void* src, unsigned char* dst) {
  __builtin_amdgcn_global_load_lds((global_void)src, (lds_void)dst, 16, 0, 0);
}

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// max over the two halves of a wave / over its four 16-lane rows
__device__ __forceinline__ float max_halves(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float max_rows(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_halves(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
}
__device__ __forceinline__ float sum_halves(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Entry of the block table for token t of sequence b (entries clamped, see
// misa_kv_pages), and the pool row it makes
__device__ __forceinline__ int table_entry(const AttnArgs& a, int b, int t) {
  const uint32_t p = a.page_shift >= 0 ? (uint32_t)t >> a.page_shift : (uint32_t)t / (uint32_t)a.page_keys;
  return a.table[(int64_t)b * a.max_pages + p];
}
__device__ __forceinline__ int pool_row(const AttnArgs& a, int entry, int t) {
  const uint32_t in = a.page_shift >= 0 ? (uint32_t)t & (uint32_t)(a.page_keys - 1) : (uint32_t)t % (uint32_t)a.page_keys;
  const int e = min(max(entry, 0), a.n_pages - 1);
  return e * a.page_keys + (int)in;   // below 2^31: the ABI bounds the pool
}

// Sequence b's new tokens t0 .. t0+m-1 (m: those within n_tokens), the position
// of the first, and its readable length.
struct SeqSpan {
  int t0, m;
  int64_t pos0;
  int len;
};
__device__ __forceinline__ SeqSpan seq_span(const AttnArgs& a, int b) {
  const int64_t s = a.q_start[b], e = a.q_start[b + 1], n = a.n_tokens;
  const int64_t kv = max(a.kv_lens[b], 0);
  SeqSpan r;
  const int64_t t0 = min(max(s, (int64_t)0), n);
  r.t0 = (int)t0;
  r.m = (int)max((int64_t)0, min(e, n) - t0);
  r.pos0 = kv - (e - s);
  r.len = (int)min(kv, a.max_pages * a.page_keys);
  return r;
}

// The sequence of token t (q_start[0] <= t < q_start[n_seq]): 64 lanes probe at
// a time.  Uniform.
__device__ __forceinline__ int seq_of_token(const AttnArgs& a, int64_t t, int lane) {
  int lo = 0, n = a.n_seq;   // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int at = lo + lane * step;
    const uint64_t m = __ballot(lane * step < n && a.q_start[min(at, a.n_seq)] <= t);
    const int j = max(63 - (int)__builtin_clzll(m | 1), 0);   // last probe at or before t
    n = min(step, n - j * step);
    lo += j * step;
  }
  return lo;
}

// -scale is folded into the sign of q, so that a maximum of scores is a maximum
// of scaled scores
__device__ __forceinline__ bf16x8 load_q(const uint16_t* p, uint32_t flip) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  return as_bf16x8(make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip));
}

// What a launch adds to the arguments
struct AttnLaunch {
  int n_units;      // row tiles (attn_tile), or sequences / tokens (attn_wave)
  int n_splits;     // key splits of a unit
  int rows_min;     // dense: attn_tile takes sequences with more rows than this, attn_wave the others
  float* part_o;    // n_splits > 1: unnormalised outputs [unit][kv head][split][row][D]
  float2* part_ml;  // and (maximum, sum) of each
};

// Dense row tiles of BM rows, numbered over the sequences with more than
// rows_min rows: tile -> sequence and first row.  64 lanes take four sequences
// each at a time.  False: no such tile.  Uniform.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int G, int rows_min, int BM, int tile, int lane, int* b_out,
                                          int* r0_out) {
  int64_t base = 0;
  for (int b0 = 0; b0 < a.n_seq; b0 += 256) {
    int c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = b0 + lane * 4 + i;
      c[i] = 0;
      if (b < a.n_seq) {
        const int64_t n = a.n_tokens;
        const int64_t t0 = min(max((int64_t)a.q_start[b], (int64_t)0), n);
        const int64_t rows = max((int64_t)0, min((int64_t)a.q_start[b + 1], n) - t0) * G;
        c[i] = rows > rows_min ? (int)((rows + BM - 1) / BM) : 0;
      }
      sum += c[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int x = __shfl_up(inc, o);
      if (lane >= o) inc += x;
    }
    const int total = __builtin_amdgcn_readlane(inc, 63);
    if (tile < base + total) {
      const int rel = (int)(tile - base);
      const uint64_t m = __ballot(inc > rel);
      const int src = (int)__builtin_ctzll(m);
      int left = rel - (inc - sum), i = 0;   // valid on lane src
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (i == k && left >= c[k]) {
          left -= c[k];
          i = k + 1;
        }
      *b_out = b0 + src * 4 + __builtin_amdgcn_readlane(i, src);
      *r0_out = __builtin_amdgcn_readlane(left, src) * BM;
      return true;
    }
    base += total;
  }
  return false;
}

// The splits of one output row: partial rows pr, pr + step, ...; out_row is the
// row of out and lse.  Lane s holds split s's weight, then every lane D / 64
// output elements.  Fixed order.
template <int D>
__device__ __forceinline__ void join_row(const AttnArgs& a, const AttnLaunch& L, int64_t pr, int64_t step, int64_t out_row,
                                         int lane) {
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < L.n_splits) ml = L.part_ml[pr + lane * step];
  float top = ml.y > 0.f ? ml.x : -INFINITY;
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float w = ml.y > 0.f ? exp2_raw(ml.x - top) : 0.f;
  float sum = w * ml.y;
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) sum += __shfl_xor(sum, x);
  constexpr int E = D / kWave;
  float o[E] = {};
  for (int s = 0; s < L.n_splits; ++s) {
    const float ws = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), s));
    if (ws == 0.f) continue;   // an empty split wrote no output
    const float* src = L.part_o + (pr + s * step) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(ws, src[e], o[e]);
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  uint16_t* dst = a.out + out_row * D + lane * E;
  if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = pk_bf16(o[0] * inv, o[1] * inv);
  else dst[0] = (uint16_t)(pk_bf16(o[0] * inv, 0.f) & 0xFFFFu);
  if (a.lse != nullptr && lane == 0) a.lse[out_row] = sum > 0.f ? (top + __log2f(sum)) * kLn2 : -INFINITY;
}

}  // namespace misa
