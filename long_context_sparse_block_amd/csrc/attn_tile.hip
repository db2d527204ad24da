// Attention of many query rows: a workgroup of NW waves takes 32 NW rows of one
// kv head, 32 a wave, and walks the keys in tiles of 64 that the waves stage
// together in LDS (double-buffered, one barrier a tile).
//
// A tile of a wave is 16 + 16 (D = 128) v_mfma_f32_32x32x16_bf16, fed by 16
// 16-byte LDS reads of K and 32 transposing 8-byte reads of V; the running
// maximum and sum of the softmax stay in one lane pair per row.  The
// output is rescaled only when a row's maximum has grown by more than 2^8 since
// the last time (the weights stay below 2^8, well inside bf16 and fp32).
//
// Bound by arithmetic: MFMA 48% and the vector unit 45% of a CU's time, one after
// the other (2048 tokens over 32K keys, 32 / 8 heads of 128: 1.07-1.15 ms by card, 930
// to 1000 TFLOP/s where the library's product reaches 1327).  At head_dim 64 over
// e4m3 pages the vector unit is the bound (70%: exponentials and scales; 9
// sequences of 0..515 new tokens over up to 5003 keys, 20 / 4 heads: 78-98 us a call).
// The 2048 tokens over e4m3 pages 1.14 ms, with heads of 64 0.63 ms (850 TFLOP/s),
// e4m3 0.73 (732).
// The weights enter the second product as one bf16 each (half a step, 2^-8, of a
// weight; a row's error is then about sqrt 2 of its output's own rounding).  A
// second part, what the rounding left, is another 16 matrix instructions a tile,
// and not hidden even where loads bound the kernel: over selected tokens, 64 x 2048
// picks of 64 / 1 heads of 128 26.4 -> 27.8 us, 1000 x 2048 146 -> 169, of 128 / 1
// heads 172 -> 214.
// 32 rows a wave: with 64, or with scores formed a tile ahead, the registers
// leave one wave a SIMD, and both were slower (1.17 to 1.6 ms).  NW = 2 where a
// unit has at most 64 rows: half the rows of 4 would be empty.
#include "attn_device.h"

namespace misa {

namespace {
constexpr int kBN = 64;          // keys of a tile
constexpr int kMfma = 0x8, kDsRead = 0x100;   // instruction classes of sched_group_barrier

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
__global__ void __launch_bounds__(NW * kWave, D == 64 ? 3 : 2) k_attn_tile(const AttnArgs a, const AttnLaunch L) {
  constexpr int NT = NW * kWave, BM = NW * 32;
  constexpr int RB = D * 2;            // bytes of a bf16 row
  constexpr int P = D / 8;             // its 16-byte pieces
  constexpr int RPI = kWave / P;       // rows of one wave-wide 16-byte load
  constexpr int kLoads = kBN / RPI / NW;
  constexpr int KS = D / 16;           // MFMA steps of a dot product
  constexpr int DB = D / 32;           // 32-wide blocks of the output
  constexpr int PC = D / 16;           // 16-byte pieces of a row of e4m3 codes
  __shared__ __attribute__((aligned(16))) unsigned char s_k0[kBN * RB], s_k1[kBN * RB], s_v0[kBN * RB], s_v1[kBN * RB];
  __shared__ __attribute__((aligned(16))) float s_ks0[kBN], s_ks1[kBN], s_vs0[kBN], s_vs1[kBN];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, c32 = lane & 31;
  const int G = a.n_heads / a.n_kv_heads;

  const Place at = place_of(L, a.n_kv_heads, blockIdx.x, SEL ? 31 : 3);
  const int split = at.split, g = at.g;
  int unit = at.unit;
  int b, r0, nrows, tok0;      // sequence, first row, its rows in all, its first token
  int64_t pos0;                // position of tok0
  int kend, kfull;             // keys some row sees, keys every row sees
  int jt0, jt1;                // the tiles of this split
  int in_use = 1;              // its unit's splits in use
  auto range = [&](const DenseScan& w) __attribute__((always_inline)) {
    const int n = (kend + kBN - 1) / kBN;
    const int per = split_tiles(w, L, n, &in_use);
    jt0 = split * per;
    jt1 = min(n, jt0 + per);
  };
  int pick0 = 0, pick1 = 0, pick2 = 0;   // SEL: this lane's listed tokens of the first three tiles
  if (SEL) {
    const int sub = (G + BM - 1) / BM;
    tok0 = unit / sub;
    r0 = (unit % sub) * BM;
    nrows = G;
    kend = a.topk;
    range(DenseScan{0.f, 0, 0, 0});
    // on their way while the sequence is looked up
    pick0 = pick(a, tok0, jt0 * kBN + lane);
    pick1 = pick(a, tok0, jt0 * kBN + kBN + lane);
    pick2 = pick(a, tok0, jt0 * kBN + 2 * kBN + lane);
    SeqSpan sp;
    if (!seq_of_token(a, tok0, lane, &b, &sp)) return;
    pos0 = sp.pos0 + (tok0 - sp.t0);
    kfull = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + 1));   // tokens the row may list
    if (kfull == 0) jt1 = jt0;
  } else {
    unit = L.n_units - 1 - unit;   // the longest prefixes of a prompt first
    SeqSpan sp;
    DenseScan scan;
    const bool tell = L.n_splits > 1 && split == 0 && g == 0 && tid == 0;   // the join's directions
    if (!find_unit<true, kBN, D>(a, L, G, BM, unit, lane, &sp, &b, &r0, &scan)) {
      if (tell) L.unit_info[unit] = make_int4(0, 0, 0, 0);
      return;
    }
    tok0 = sp.t0;
    nrows = sp.m * G;
    pos0 = sp.pos0;
    const int last = (min(r0 + BM, nrows) - 1) / G, first = r0 / G;
    kend = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + last + 1));
    kfull = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + first + 1));
    range(scan);
    if (tell) L.unit_info[unit] = make_int4(tok0, r0, nrows, in_use);
    if (split >= in_use) return;
  }

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
  auto token_at = [&](int jt) __attribute__((always_inline)) -> int {
    const int j = jt * kBN + lane;
    return SEL ? pick(a, tok0, j) : min(j, kend - 1);
  };
  using Stage = Fp8Stage<D, NT>;
  // Lane k of every wave knows where key k's pool row starts (bytes); a load's
  // lanes fetch that from the lane of their row.  Which piece of the row a lane
  // moves is the same for all its loads where their rows are 16 apart (every
  // other one where they are 8 apart), so the rest of the address is fixed.
  const int64_t row_bytes = (int64_t)a.n_kv_heads * D * (FP8 ? 1 : 2);
  const int lrow = FP8 ? tid / PC : wave * RPI + lane / P;   // row of the first load
  const int lpiece = FP8 ? tid % PC : (lane % P) ^ swizzle<D>(lrow);
  const char* const kl = static_cast<const char*>(a.k) + g * D * (FP8 ? 1 : 2) + lpiece * 16;
  const char* const vl = static_cast<const char*>(a.v) + g * D * (FP8 ? 1 : 2) + lpiece * 16;
  constexpr int kStepRows = FP8 ? NT / PC : NW * RPI;        // rows between a lane's loads
  static_assert(kStepRows % 16 == 0 || (kStepRows == 8 && !FP8), "a lane's piece and its place in LDS repeat");
  const int lodd = kStepRows % 16 == 0 ? 0 : (((lane % P) ^ swizzle<D>(lrow + 8)) - lpiece) * 16;   // of odd loads
  auto fetch = [&](int64_t off, int from) __attribute__((always_inline)) -> int64_t {
    const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)off, from), hi = (uint32_t)__shfl((int)(off >> 32), from);
    return (int64_t)(((uint64_t)hi << 32) | lo);
  };
  // a tile towards LDS: bf16 straight there, e4m3 codes into registers, from
  // which land() widens them
  auto issue = [&](int row_of, unsigned char* dk, unsigned char* dv, Stage& st) __attribute__((always_inline)) {
    const int64_t mine = (int64_t)row_of * row_bytes;
    constexpr int N = FP8 ? Stage::kLoads : kLoads;
    int64_t off[N];
#pragma unroll
    for (int u = 0; u < N; ++u) off[u] = fetch(mine, (lrow + u * kStepRows) & 63) + (kStepRows == 8 && (u & 1) ? lodd : 0);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if constexpr (!FP8) {
        load_lds16(kl + off[u], dk + (u * NW + wave) * RPI * RB);
        load_lds16(vl + off[u], dv + (u * NW + wave) * RPI * RB);
      } else {
        st.k[u] = *reinterpret_cast<const uint4*>(kl + off[u]);
        st.v[u] = *reinterpret_cast<const uint4*>(vl + off[u]);
      }
    }
    if constexpr (FP8) {
      if (wave == 0) st.scale = a.k_scale[(int64_t)row_of * a.n_kv_heads + g];
      if (wave == NW - 1 && wave != 0) st.scale = a.v_scale[(int64_t)row_of * a.n_kv_heads + g];
    }
  };
  const int lf = swizzle<D>(lrow);
  const int land0 = lrow * RB + (((2 * lpiece) ^ lf) << 4), land1 = lrow * RB + (((2 * lpiece + 1) ^ lf) << 4);
  auto land = [&](const Stage& st, unsigned char* dk, unsigned char* dv, float* dks, float* dvs) __attribute__((always_inline)) {
    if constexpr (FP8) {
#pragma unroll
      for (int u = 0; u < Stage::kLoads; ++u) {
        auto put = [&](unsigned char* d, uint4 x) __attribute__((always_inline)) {
          const uint2 w0 = e4m3x4_to_bf16x4(x.x), w1 = e4m3x4_to_bf16x4(x.y);
          const uint2 w2 = e4m3x4_to_bf16x4(x.z), w3 = e4m3x4_to_bf16x4(x.w);
          *reinterpret_cast<uint4*>(d + u * kStepRows * RB + land0) = make_uint4(w0.x, w0.y, w1.x, w1.y);
          *reinterpret_cast<uint4*>(d + u * kStepRows * RB + land1) = make_uint4(w2.x, w2.y, w3.x, w3.y);
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
                     uint64_t mask) __attribute__((always_inline)) {
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
    // six reads ahead of the products (left alone, the compiler waits for each)
    __builtin_amdgcn_sched_group_barrier(kDsRead, 6, 0);
#pragma unroll
    for (int i = 0; i < 2 * KS - 6; ++i) {
      __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, 6, 0);
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
      float sum[4] = {p[0], p[1], p[2], p[3]};
#pragma unroll
      for (int e = 4; e < 16; ++e) sum[e & 3] += p[e];
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
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int db = 0; db < DB; ++db) {
        const int x = (db ^ vx) << 6;
        const uint2 lo = lds_read_tr(sv + t * 16 * RB + v_base[0] + x), hi = lds_read_tr(sv + t * 16 * RB + v_base[1] + x);
        o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y)), pf[t], o[db], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_group_barrier(kDsRead, 8, 0);
#pragma unroll
    for (int i = 0; i < 4 * DB - 4; ++i) {
      __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kDsRead, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, 4, 0);
  };

  if (jt0 < jt1) {
    const int last = jt1 - 1;
    // An absent entry (a weight of 0) reads the tile's first listed token instead,
    // whose value the row sees anyway; a tile without one is skipped.
    auto look = [&](int t, uint64_t& mask) __attribute__((always_inline)) -> int {
      if (!SEL) return t;
      const bool in = t >= 0 && t < kfull;
      mask = __ballot(in);
      const int first = mask != 0 ? __builtin_amdgcn_readlane(t, (int)__builtin_ctzll(mask)) : 0;
      return in ? t : first;
    };
    uint64_t m0 = ~0ull, m1 = ~0ull, m2 = ~0ull;   // of this tile and the next two
    const int t0 = look(SEL ? pick0 : token_at(jt0), m0);
    const int t1 = look(SEL ? pick1 : token_at(min(jt0 + 1, last)), m1);
    const int e0 = table_entry(a, b, t0), e1 = table_entry(a, b, t1);
    if constexpr (!FP8) {
      // One tile ahead, straight into the other buffer; look-ups run a tile
      // further ahead each (the table entry, then the listed token).
      Stage none;
      issue(pool_row(a, e0, t0), s_k0, s_v0, none);
      int tok_n = t1, ent_n = e1, tok_nn = SEL ? pick2 : token_at(min(jt0 + 2, last));
      auto step = [&](int jt, const unsigned char* ck, const unsigned char* cv, unsigned char* nk, unsigned char* nv) __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();   // tile jt is in LDS, and nobody reads the other buffer any more
        if (jt + 1 < jt1) {
          issue(pool_row(a, ent_n, tok_n), nk, nv, none);
          tok_n = look(tok_nn, m2);
          ent_n = table_entry(a, b, tok_n);
          tok_nn = token_at(min(jt + 3, last));
        }
        if (!SEL || m0 != 0) compute(ck, cv, s_ks0, s_vs0, jt, m0);
        m0 = m1;
        m1 = m2;
      };
      for (int jt = jt0; jt < jt1; jt += 2) {
        step(jt, s_k0, s_v0, s_k1, s_v1);
        if (jt + 1 < jt1) step(jt + 1, s_k1, s_v1, s_k0, s_v0);
      }
    } else {
      // Codes two tiles ahead in registers, widened into the other buffer after
      // the tile before is done with.  Loads return in order, so a step's
      // look-ups go out before its codes: waiting for them then waits for no
      // codes but the oldest.  Near the end the last tile is loaded again: loads
      // behind a branch would make the compiler wait for all of them.
      Stage sa, sb;
      int tok_n = look(SEL ? pick2 : token_at(min(jt0 + 2, last)), m2);
      int ent_n = table_entry(a, b, tok_n);
      int tok_nn = token_at(min(jt0 + 3, last));
      issue(pool_row(a, e0, t0), nullptr, nullptr, sa);
      __builtin_amdgcn_sched_barrier(0);   // in this order
      issue(pool_row(a, e1, t1), nullptr, nullptr, sb);
      __builtin_amdgcn_sched_barrier(0);
      land(sa, s_k0, s_v0, s_ks0, s_vs0);
      auto step = [&](int jt, const unsigned char* ck, const unsigned char* cv, const float* cks, const float* cvs,
                      unsigned char* nk, unsigned char* nv, float* nks, float* nvs, Stage& free, const Stage& next) __attribute__((always_inline)) {
        __syncthreads();   // tile jt is in LDS, and nobody reads the other buffer any more
        uint64_t m3 = ~0ull;
        const int row = pool_row(a, ent_n, tok_n);
        tok_n = look(tok_nn, m3);
        ent_n = table_entry(a, b, tok_n);
        tok_nn = token_at(min(jt + 4, last));
        issue(row, nullptr, nullptr, free);
        if (!SEL || m0 != 0) compute(ck, cv, cks, cvs, jt, m0);
        land(next, nk, nv, nks, nvs);
        m0 = m1;
        m1 = m2;
        m2 = m3;
      };
      for (int jt = jt0;;) {   // (one way back to the top, for the compiler's count of loads under way)
        step(jt, s_k0, s_v0, s_ks0, s_vs0, s_k1, s_v1, s_ks1, s_vs1, sa, sb);
        if (++jt >= jt1) break;
        step(jt, s_k1, s_v1, s_ks1, s_vs1, s_k0, s_v0, s_ks0, s_vs0, sb, sa);
        if (++jt >= jt1) break;
      }
    }
  }

  l = sum_halves(l);
  // o[db][4 j + i] of the lane: element db 32 + 8 j + 4 h + i of row r
  if (in_use == 1) {
    if (!live) return;
    const float inv = l != 0.f ? 1.f / l : 0.f;
    uint16_t* dst = a.out + (qrow * a.n_heads + qh) * D;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint2*>(dst + db * 32 + 8 * j + 4 * h) =
            make_uint2(pk_bf16(o[db][4 * j] * inv, o[db][4 * j + 1] * inv), pk_bf16(o[db][4 * j + 2] * inv, o[db][4 * j + 3] * inv));
    if (a.lse != nullptr && h == 0) a.lse[qrow * a.n_heads + qh] = l != 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
    return;
  }
  if (!live) return;
  const PartPlace part = part_place<SEL>(L, a.n_kv_heads, G, BM, g, unit, tok0, r0, nrows);
  const int64_t pr = part.begin + split * part.step + wave * 32 + c32;
  if (h == 0) L.part_ml[pr] = make_float2(m, l);
  if (l != 0.f) {
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(L.part_o + pr * D + db * 32 + 8 * j + 4 * h) =
            f32x4{o[db][4 * j], o[db][4 * j + 1], o[db][4 * j + 2], o[db][4 * j + 3]};
  }
}

template <int D, bool FP8, bool SEL>
static hipError_t launch_nw(const AttnArgs& a, const AttnLaunch& L, int NW, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)L.n_units * L.n_splits * a.n_kv_heads));
  if (NW == 2) hipLaunchKernelGGL((k_attn_tile<D, FP8, SEL, 2>), grid, dim3(128), 0, st, a, L);
  else hipLaunchKernelGGL((k_attn_tile<D, FP8, SEL, 4>), grid, dim3(256), 0, st, a, L);
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
