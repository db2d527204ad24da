// Attention of many query rows: a workgroup of NW waves takes 32 NW rows of one
// kv head, 32 a wave, and walks the keys in tiles of 64 that the waves stage
// together in LDS (double-buffered, one barrier a tile).
//
// A tile of a wave is 16 + 16 (D = 128) v_mfma_f32_32x32x16_bf16, fed by 16
// 16-byte LDS reads of K and 32 transposing 8-byte reads of V; the running
// maximum and sum of the softmax stay in one lane pair per row.  The
// output is rescaled only when a row's maximum has grown by more than 2^8 since
// the last time (the weights stay below 2^8, well inside bf16 and fp32).
#include "attn_device.h"

namespace misa {

namespace {
constexpr int kBN = 64;          // keys of a tile
constexpr float kGrow = 8.f;     // log2 of the growth that forces a rescale

// e4m3 codes of the tile, 16 bytes a load, on their way to bf16 rows in LDS
template <int D, int NT>
struct Fp8Stage {
  static constexpr int kPieces = D / 16;                  // 16-byte pieces of a row of codes
  static constexpr int kLoads = kBN * kPieces / NT;       // a thread's, for K and for V
  uint4 k[kLoads], v[kLoads];
  float scale;
};
}  // namespace

template <int D, bool FP8, bool SEL, int NW>
__global__ void __launch_bounds__(NW * kWave, 2) k_attn_tile(const AttnArgs a, const AttnLaunch L) {
  constexpr int NT = NW * kWave, BM = NW * 32;
  constexpr int RB = D * 2;            // bytes of a bf16 row
  constexpr int P = D / 8;             // its 16-byte pieces
  constexpr int RPI = kWave / P;       // rows of one wave-wide 16-byte load
  constexpr int kLoads = kBN / RPI / NW;
  constexpr int KS = D / 16;           // MFMA steps of a dot product
  constexpr int DB = D / 32;           // 32-wide blocks of the output
  __shared__ __attribute__((aligned(16))) unsigned char s_k0[kBN * RB], s_k1[kBN * RB], s_v0[kBN * RB], s_v1[kBN * RB];
  __shared__ __attribute__((aligned(16))) float s_ks0[kBN], s_ks1[kBN], s_vs0[kBN], s_vs1[kBN];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, c32 = lane & 31;
  const int G = a.n_heads / a.n_kv_heads;

  // unit order: kv head, split, row tile (an XCD then walks row tiles of the
  // same keys), the tiles with the longest prefixes first
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int rest = (int)(id / L.n_units);
  int unit = (int)(id % L.n_units);
  const int split = rest % L.n_splits, g = rest / L.n_splits;
  int b, r0, nrows, tok0;      // sequence, first row, its rows in all, its first token
  int64_t pos0;                // position of tok0
  int kend, kfull;             // keys some row sees, keys every row sees
  if (SEL) {
    const int sub = (G + BM - 1) / BM;
    tok0 = unit / sub;
    r0 = (unit % sub) * BM;
    if (tok0 >= a.q_start[a.n_seq] || tok0 < a.q_start[0]) return;
    b = seq_of_token(a, tok0, lane);
    const SeqSpan sp = seq_span(a, b);
    nrows = G;
    pos0 = sp.pos0 + (tok0 - sp.t0);
    kfull = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + 1));   // tokens the row may list
    kend = kfull > 0 ? a.topk : 0;
  } else {
    unit = L.n_units - 1 - unit;
    if (!find_tile(a, G, L.rows_min, BM, unit, lane, &b, &r0)) return;
    const SeqSpan sp = seq_span(a, b);
    tok0 = sp.t0;
    nrows = sp.m * G;
    pos0 = sp.pos0;
    const int last = (min(r0 + BM, nrows) - 1) / G, first = r0 / G;
    kend = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + last + 1));
    kfull = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + first + 1));
  }
  const int n_tiles_all = (kend + kBN - 1) / kBN;
  const int per = (n_tiles_all + L.n_splits - 1) / L.n_splits;
  const int jt0 = split * per, jt1 = min(n_tiles_all, jt0 + per);

  // this lane's query row (rows past the end repeat the last one and are not written)
  const int r = r0 + wave * 32 + c32;
  const bool live = r < nrows;
  const int rc = min(r, nrows - 1);
  const int qi = SEL ? 0 : rc / G, qh = g * G + (SEL ? rc : rc - qi * G);
  const int64_t qrow = (int64_t)tok0 + qi;
  const int64_t rpos = SEL ? 0 : pos0 + qi;
  const int vis = SEL ? 0 : (int)max((int64_t)-1, min((int64_t)kend, rpos + 1));   // the row sees keys below vis

  const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
  const float sc = fmaxf(fabsf(a.scale_log2), 1e-30f);
  bf16x8 qf[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) qf[ks] = load_q(a.q + qrow * a.q_st + qh * a.q_sh + ks * 16 + h * 8, flip);

  // Staging.  Lane k of every wave looks up key k of a tile two tiles ahead:
  // the listed token (SEL) three tiles ahead, its table entry two, so that no
  // load is waited for in the iteration that issues it.
  const int64_t row_stride = (int64_t)a.n_kv_heads * D;   // elements of a pool row
  auto token_at = [&](int jt) -> int {
    const int j = jt * kBN + lane;
    if (SEL) return j < a.topk ? a.idx[qrow * a.topk + j] : -1;
    return min(j, kend - 1);
  };
  auto clamp_tok = [&](int t) -> int { return SEL ? (t >= 0 && t < kfull ? t : 0) : t; };
  int tok_n = 0, ent_n = 0;       // tile in flight: token, table entry
  int row_c = 0;                  // pool row of the next tile's key `lane`
  uint64_t mask_n = ~0ull, mask_c = ~0ull;
  Fp8Stage<D, NT> st;

  auto issue = [&](unsigned char* dk, unsigned char* dv) {   // tile of row_c
    if constexpr (!FP8) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int base = (u * NW + wave) * RPI;
        const int row = base + lane / P;
        const int64_t off = ((int64_t)__shfl(row_c, row) * row_stride + g * D) * 2 + ((lane % P) ^ swizzle<D>(row)) * 16;
        load_lds16(static_cast<const char*>(a.k) + off, dk + base * RB);
        load_lds16(static_cast<const char*>(a.v) + off, dv + base * RB);
      }
    } else {
      constexpr int PC = Fp8Stage<D, NT>::kPieces;
#pragma unroll
      for (int u = 0; u < Fp8Stage<D, NT>::kLoads; ++u) {
        const int i = u * NT + tid;
        const int64_t off = (int64_t)__shfl(row_c, i / PC) * row_stride + g * D + (i % PC) * 16;
        st.k[u] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) + off);
        st.v[u] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.v) + off);
      }
      if (wave == 0) st.scale = a.k_scale[(int64_t)row_c * a.n_kv_heads + g];
      if (wave == NW - 1 && wave != 0) st.scale = a.v_scale[(int64_t)row_c * a.n_kv_heads + g];
    }
  };
  auto land = [&](unsigned char* dk, unsigned char* dv, float* dks, float* dvs) {   // FP8: registers -> LDS
    if constexpr (FP8) {
      constexpr int PC = Fp8Stage<D, NT>::kPieces;
#pragma unroll
      for (int u = 0; u < Fp8Stage<D, NT>::kLoads; ++u) {
        const int i = u * NT + tid, row = i / PC, c = 2 * (i % PC);
        const int f = swizzle<D>(row);
        auto put = [&](unsigned char* d, uint4 x) {
          const uint2 w0 = e4m3x4_to_bf16x4(x.x), w1 = e4m3x4_to_bf16x4(x.y);
          const uint2 w2 = e4m3x4_to_bf16x4(x.z), w3 = e4m3x4_to_bf16x4(x.w);
          *reinterpret_cast<uint4*>(d + row * RB + ((c ^ f) << 4)) = make_uint4(w0.x, w0.y, w1.x, w1.y);
          *reinterpret_cast<uint4*>(d + row * RB + (((c + 1) ^ f) << 4)) = make_uint4(w2.x, w2.y, w3.x, w3.y);
        };
        put(dk, st.k[u]);
        put(dv, st.v[u]);
      }
      if (wave == 0) dks[lane] = st.scale;
      if (wave == NW - 1 && wave != 0) dvs[lane] = st.scale;
    }
  };

  f32x16 o[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[i][e] = 0.f;
  float m = -INFINITY, l = 0.f;

  // LDS addresses of the lane's reads (see swizzle)
  const int f = swizzle<D>(c32);
  const int k_base = c32 * RB + ((h ^ f) << 4);
  const int vr = (lane & 15) >> 2;                                       // row of four
  const int vc = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);              // piece of the 32-wide block
  const int vx = D == 128 ? vr : vr >> 1;                                // the swizzle's high bits
  int v_base[2];
#pragma unroll
  for (int e2 = 0; e2 < 2; ++e2)
    v_base[e2] = (8 * e2 + 4 * h + vr) * RB + ((vc ^ (2 * e2 + h)) << 4) + (lane & 1) * 8;

  auto compute = [&](const unsigned char* sk, const unsigned char* sv, const float* sks, const float* svs, int jt,
                     uint64_t mask) {
    f32x16 s[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[kb][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const bf16x8 kf = as_bf16x8(*reinterpret_cast<const uint4*>(sk + kb * 32 * RB + (k_base ^ (ks << 5))));
        s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[ks], s[kb], 0, 0, 0);
      }
    }
    // key of s[kb][4 j + i]: kb 32 + 8 j + 4 h + i
    if constexpr (FP8) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 w = *reinterpret_cast<const f32x4*>(sks + kb * 32 + 8 * j + 4 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[kb][4 * j + i] *= w[i];
        }
    }
    if (SEL) {
      if (mask != ~0ull) {
        const uint32_t mw[2] = {(uint32_t)mask >> (4 * h), (uint32_t)(mask >> 32) >> (4 * h)};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!((mw[kb] >> (8 * (e >> 2) + (e & 3))) & 1)) s[kb][e] = -INFINITY;
      }
    } else if ((jt + 1) * kBN > kfull) {
      const int lim = vis - jt * kBN - 4 * h;   // the row sees the tile's keys below this
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (kb * 32 + 8 * (e >> 2) + (e & 3) >= lim) s[kb][e] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[kb][e]);
    top = max_halves(top) * sc;
    if (__any(top > m + kGrow)) {   // (m = -inf at first)
      const float mn = fmaxf(m, top);
      const float keep = mn == -INFINITY ? 1.f : exp2_raw(m - mn);
      m = mn;
      l *= keep;
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] *= keep;
    }
    const float mu = m == -INFINITY ? 0.f : m;
    bf16x8 pf[4];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float p[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) p[e] = exp2_raw(__builtin_fmaf(s[kb][e], sc, -mu));
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 16; ++e) sum[e & 3] += p[e];
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if constexpr (FP8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 w = *reinterpret_cast<const f32x4*>(svs + kb * 32 + 8 * j + 4 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) p[4 * j + i] *= w[i];
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
        pf[2 * kb + q] = as_bf16x8(make_uint4(pk_bf16(p[8 * q], p[8 * q + 1]), pk_bf16(p[8 * q + 2], p[8 * q + 3]),
                                              pk_bf16(p[8 * q + 4], p[8 * q + 5]), pk_bf16(p[8 * q + 6], p[8 * q + 7])));
    }
#pragma unroll
    for (int db = 0; db < DB; ++db) {
      const int x = (db ^ vx) << 6;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint2 lo = lds_read_tr(sv + t * 16 * RB + v_base[0] + x), hi = lds_read_tr(sv + t * 16 * RB + v_base[1] + x);
        o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y)), pf[t], o[db], 0, 0, 0);
      }
    }
  };

  if (jt0 < jt1) {
    // first tile's rows, second tile's entries, third tile's tokens
    const int last = jt1 - 1;
    int t = token_at(jt0);
    if (SEL) mask_n = __ballot(t >= 0 && t < kfull);
    t = clamp_tok(t);
    row_c = pool_row(a, table_entry(a, b, t), t);
    uint64_t mask_first = mask_n;
    issue(s_k0, s_v0);
    land(s_k0, s_v0, s_ks0, s_vs0);
    tok_n = token_at(min(jt0 + 1, last));
    if (SEL) mask_n = __ballot(tok_n >= 0 && tok_n < kfull);
    tok_n = clamp_tok(tok_n);
    ent_n = table_entry(a, b, tok_n);
    int tok_nn = token_at(min(jt0 + 2, last));
    mask_c = mask_first;
    auto step = [&](int jt, unsigned char* ck, unsigned char* cv, float* cks, float* cvs, unsigned char* nk,
                    unsigned char* nv, float* nks, float* nvs) {
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();   // tile jt is in LDS, and nobody reads the other buffer any more
      const bool more = jt + 1 < jt1;
      const uint64_t mask_next = mask_n;
      if (more) {
        row_c = pool_row(a, ent_n, tok_n);
        issue(nk, nv);
        if (SEL) mask_n = __ballot(tok_nn >= 0 && tok_nn < kfull);
        tok_n = clamp_tok(tok_nn);
        ent_n = table_entry(a, b, tok_n);
        tok_nn = token_at(min(jt + 3, last));
      }
      compute(ck, cv, cks, cvs, jt, mask_c);
      if (more) land(nk, nv, nks, nvs);
      mask_c = mask_next;
    };
    for (int jt = jt0; jt < jt1; jt += 2) {
      step(jt, s_k0, s_v0, s_ks0, s_vs0, s_k1, s_v1, s_ks1, s_vs1);
      if (jt + 1 < jt1) step(jt + 1, s_k1, s_v1, s_ks1, s_vs1, s_k0, s_v0, s_ks0, s_vs0);
    }
  }

  l = sum_halves(l);
  // o[db][4 j + i] of the lane: element db 32 + 8 j + 4 h + i of row r
  if (L.n_splits == 1) {
    if (!live) return;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t* dst = a.out + (qrow * a.n_heads + qh) * D;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint2*>(dst + db * 32 + 8 * j + 4 * h) =
            make_uint2(pk_bf16(o[db][4 * j] * inv, o[db][4 * j + 1] * inv), pk_bf16(o[db][4 * j + 2] * inv, o[db][4 * j + 3] * inv));
    if (a.lse != nullptr && h == 0) a.lse[qrow * a.n_heads + qh] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
    return;
  }
  const int64_t pr = (((int64_t)unit * a.n_kv_heads + g) * L.n_splits + split) * BM + wave * 32 + c32;
  if (h == 0) L.part_ml[pr] = make_float2(m, l);
  if (l > 0.f) {
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(L.part_o + pr * D + db * 32 + 8 * j + 4 * h) =
            f32x4{o[db][4 * j], o[db][4 * j + 1], o[db][4 * j + 2], o[db][4 * j + 3]};
  }
}

// The splits of a row joined: one wave a row, lane s first holds split s's
// (maximum, sum), then D / 64 output elements.  Fixed order, so the same call
// gives the same bits.
template <int D, bool SEL>
__global__ void __launch_bounds__(256) k_attn_tile_join(const AttnArgs a, const AttnLaunch L, int BM) {
  const int lane = threadIdx.x & 63;
  const int unit = blockIdx.x, g = blockIdx.y;
  const int G = a.n_heads / a.n_kv_heads;
  const int rr = blockIdx.z * 4 + (threadIdx.x >> 6);   // row of the tile
  int b, r0, nrows, tok0;
  if (SEL) {
    const int sub = (G + BM - 1) / BM;
    tok0 = unit / sub;
    r0 = (unit % sub) * BM;
    if (tok0 >= a.q_start[a.n_seq] || tok0 < a.q_start[0]) return;
    nrows = G;
  } else {
    if (!find_tile(a, G, L.rows_min, BM, unit, lane, &b, &r0)) return;
    const SeqSpan sp = seq_span(a, b);
    tok0 = sp.t0;
    nrows = sp.m * G;
  }
  const int r = r0 + rr;
  if (r >= nrows) return;
  const int qi = SEL ? 0 : r / G, qh = g * G + (SEL ? r : r - qi * G);
  join_row<D>(a, L, (((int64_t)unit * a.n_kv_heads + g) * L.n_splits) * BM + rr, BM, ((int64_t)tok0 + qi) * a.n_heads + qh,
              lane);
}

template <int D, bool FP8, bool SEL>
static hipError_t launch_nw(const AttnArgs& a, const AttnLaunch& L, int NW, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)L.n_units * L.n_splits * a.n_kv_heads));
  if (NW == 2) hipLaunchKernelGGL((k_attn_tile<D, FP8, SEL, 2>), grid, dim3(128), 0, st, a, L);
  else hipLaunchKernelGGL((k_attn_tile<D, FP8, SEL, 4>), grid, dim3(256), 0, st, a, L);
  if (L.n_splits > 1)
    hipLaunchKernelGGL((k_attn_tile_join<D, SEL>), dim3(L.n_units, a.n_kv_heads, NW * 8), dim3(256), 0, st, a, L, NW * 32);
  return hipGetLastError();
}

hipError_t launch_attn_tile(const AttnArgs& a, const AttnLaunch& L, int D, bool fp8, int NW, hipStream_t st) {
  const bool sel = a.idx != nullptr;
  if (D == 128) {
    if (fp8) return sel ? launch_nw<128, true, true>(a, L, NW, st) : launch_nw<128, true, false>(a, L, NW, st);
    return sel ? launch_nw<128, false, true>(a, L, NW, st) : launch_nw<128, false, false>(a, L, NW, st);
  }
  if (fp8) return sel ? launch_nw<64, true, true>(a, L, NW, st) : launch_nw<64, true, false>(a, L, NW, st);
  return sel ? launch_nw<64, false, true>(a, L, NW, st) : launch_nw<64, false, false>(a, L, NW, st);
}

}  // namespace misa
