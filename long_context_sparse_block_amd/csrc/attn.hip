// Causal attention of new tokens over a paged cache (misa_attention_paged) and
// over the tokens the indexer selected (misa_attention_selected).
//
//   out = sum_s softmax_s(scale q . k[s]) v[s],   lse = log sum_s exp(scale q . k[s])
//
// One wave for each (token, query head).  Keys in runs of 64: lane l holds key
// l of the run, its score and (after the run's maximum) its weight; then the
// lanes turn to output elements, D / 64 of them each, and walk the run's
// values.  One pass over the keys with the running maximum and sum.
#include <math.h>

#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

namespace {
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
}  // namespace

// The pool row of token t of sequence b (entries clamped, see misa_kv_pages)
__device__ __forceinline__ int64_t kv_row(const AttnArgs& a, int b, int t) {
  const uint32_t p = (uint32_t)t / (uint32_t)a.page_keys;
  int64_t e = a.table[(int64_t)b * a.max_pages + min((int64_t)p, a.max_pages - 1)];
  e = e < 0 ? 0 : (e >= a.n_pages ? a.n_pages - 1 : e);
  return e * a.page_keys + (t - (int64_t)p * a.page_keys);
}

template <bool FP8>
__device__ __forceinline__ float kv_elem(const void* pool, int64_t i) {
  if constexpr (FP8) return e4m3_to_f32(static_cast<const uint8_t*>(pool)[i]);
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(pool)[i]);
}

template <int D, bool FP8, bool SEL>
__global__ void __launch_bounds__(kWave) k_attn_row(AttnArgs a) {
  __shared__ float s_q[D];
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, g = h / (a.n_heads / a.n_kv_heads);
  const int lane = threadIdx.x;
  if (t >= a.q_start[a.n_seq]) return;
  int lo = 0, hi = a.n_seq;   // last b with q_start[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int b = lo;
  const int64_t len = min((int64_t)max(a.kv_lens[b], 0), a.max_pages * a.page_keys);
  const int64_t pos = (int64_t)a.kv_lens[b] - (a.q_start[b + 1] - t);
  const int n = (int)max((int64_t)0, min(len, pos + 1));   // visible keys: tokens 0 .. n-1
  for (int d = lane; d < D; d += kWave) s_q[d] = bf16_bits_to_f32(a.q[t * a.q_st + h * a.q_sh + d]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[D / kWave] = {};
  const int count = SEL ? a.topk : n;
  for (int j0 = 0; j0 < count; j0 += kWave) {
    const int j = j0 + lane;
    int tok = SEL ? (j < count ? a.idx[t * a.topk + j] : -1) : j;
    const bool seen = tok >= 0 && tok < n && j < count;
    int64_t row = 0;
    float s = -INFINITY, vs = 1.f;
    if (seen) {
      row = kv_row(a, b, tok) * a.n_kv_heads + g;
      float acc = 0.f;
      for (int d = 0; d < D; ++d) acc = __builtin_fmaf(s_q[d], kv_elem<FP8>(a.k, row * D + d), acc);
      if (FP8) {
        acc *= a.k_scale[row];
        vs = a.v_scale[row];
      }
      s = acc * a.scale_log2;
    }
    float top = s;
    for (int x = 32; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    if (top == -INFINITY) continue;
    const float mn = fmaxf(m, top), keep = exp2f(m - mn);
    const float p = seen ? exp2f(s - mn) : 0.f;
    float sum = p;
    for (int x = 32; x >= 1; x >>= 1) sum += __shfl_xor(sum, x);
    l = l * keep + sum;
    m = mn;
    for (int i = 0; i < D / kWave; ++i) o[i] *= keep;
    const float pv = p * vs;
    for (int x = 0; x < kWave; ++x) {
      const float w = __shfl(pv, x);
      const int64_t r = __shfl(row, x);
      if (w == 0.f) continue;
      for (int i = 0; i < D / kWave; ++i)
        o[i] = __builtin_fmaf(w, kv_elem<FP8>(a.v, r * D + i * kWave + lane), o[i]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int i = 0; i < D / kWave; ++i)
    a.out[(t * a.n_heads + h) * D + i * kWave + lane] = (uint16_t)(pk_bf16(o[i] * inv, 0.f) & 0xFFFFu);
  if (a.lse != nullptr && lane == 0) a.lse[t * a.n_heads + h] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

size_t attn_workspace_bytes(const misa_attn_shape&, const misa_kv_pages&, int) { return 0; }

template <int D, bool FP8>
static void launch_rows(const AttnArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.n_tokens, (unsigned)a.n_heads);
  if (a.idx != nullptr) hipLaunchKernelGGL((k_attn_row<D, FP8, true>), grid, dim3(kWave), 0, st, a);
  else hipLaunchKernelGGL((k_attn_row<D, FP8, false>), grid, dim3(kWave), 0, st, a);
}

hipError_t launch_attention(const misa_attn_shape& s, const misa_kv_pages& pg, const uint16_t* q,
                            const int32_t* q_start, const int32_t* kv_lens, const int32_t* idx, int topk,
                            uint16_t* out, float* lse, void* ws, hipStream_t st) {
  const AttnArgs a{q, s.q_stride_token, s.q_stride_head, pg.k, pg.v, pg.k_scale, pg.v_scale, pg.block_table,
                   pg.max_pages, pg.n_pages, pg.page_keys, q_start, kv_lens, idx, topk, out, lse,
                   s.scale * kLog2e, s.n_seq, s.n_heads, s.n_kv_heads, s.n_tokens};
  const bool fp8 = pg.kdtype == MISA_K_FP8_E4M3;
  if (s.head_dim == 128) fp8 ? launch_rows<128, true>(a, st) : launch_rows<128, false>(a, st);
  else fp8 ? launch_rows<64, true>(a, st) : launch_rows<64, false>(a, st);
  return hipGetLastError();
}

}  // namespace misa
