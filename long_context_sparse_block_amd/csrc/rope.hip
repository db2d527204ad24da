// Rotary positions (misa_rope) and the write of new rows into a paged cache
// (misa_write_pages, which rotates the keys on their way).
//
// Pair j of a token at position p turns by p * inv_freq[j].  The angle is
// formed in fp64 as turns (p * inv_freq / 2 pi) and reduced by dropping its
// whole turns, so a position of 10^6 costs no precision; cos and sin are then
// those of a fraction of a turn.  They depend on (token, pair) alone: a
// workgroup takes a few tokens, forms their table once in LDS and uses it for
// every head.
//
// Both kernels are bound by HBM: each value is read once and written once, 16
// bytes a lane and access where the sizes are multiples of it.  Measured, with
// inputs that are not in the caches: 8192 tokens x 64 heads of 128 in bf16 in 50.4
// us (5.3 TB/s, a copy's rate); keys and values of 4099 tokens x 8 heads of 128
// into bf16 pages in 10.3 us (3.3 TB/s, held by the way from slot and row to the
// page: one pass of rows to a thread); 8192 index keys into e4m3 pages in 6.1 us.
// Off 16-byte pieces, one element a lane: 8192 x 32 heads of 80, 20 of them turned,
// bf16 52 us (1.6 TB/s), fp32 66 us (2.5 TB/s).  8192 x 8 + 8 heads of 128 into
// pages: bf16 16.3 us, e4m3 29.2 (fp64 angles and rotation), not turned 12.2 and
// 17.1, at an odd offset (60 values from 3 on) 25.7 and 37.1.
#include <algorithm>

#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

namespace {
constexpr int kThreads = 256;
constexpr int64_t kMaxGroups = 1 << 20;   // workgroups of a launch (it holds fewer than 2^32 threads)
constexpr double kInv2Pi = 0.15915494309189533576888;

// cos and sin of `turns` whole turns, times m.  The first rounds the reduced angle
// to fp32 (2^-25 of a half turn, 2^-23.3 in the functions): under a hundredth of a
// step of the 16-bit types it serves.
__device__ __forceinline__ float2 turn_f32(double turns, double m) {
  const float r = (float)(2.0 * (turns - __builtin_rint(turns)));   // half turns in [-1, 1]
  float s, c;
  sincospif(r, &s, &c);
  return make_float2((float)(c * m), (float)(s * m));
}
__device__ __forceinline__ double2 turn_f64(double turns, double m) {
  double s, c;
  sincospi(2.0 * (turns - __builtin_rint(turns)), &s, &c);
  return make_double2(c * m, s * m);
}

template <int DT> struct Elem;
template <> struct Elem<MISA_T_BF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float load(T x) { return bf16_bits_to_f32(x); }
  static __device__ __forceinline__ T store(float x) { return (T)(pk_bf16(x, 0.f) & 0xFFFFu); }
};
template <> struct Elem<MISA_T_FP16> {
  using T = uint16_t;
  static __device__ __forceinline__ float load(T x) { return (float)__builtin_bit_cast(_Float16, x); }
  static __device__ __forceinline__ T store(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
};
template <> struct Elem<MISA_T_FP32> {
  using T = float;
  static __device__ __forceinline__ float load(T x) { return x; }
  static __device__ __forceinline__ T store(float x) { return x; }
};

struct RopeArgs {
  const double* inv_freq;
  const int32_t* positions;
  int half, start, layout;
  double mscale;
  float sign;   // -1: the transposed rotation
};

RopeArgs rope_args(const misa_rope_spec& r) {
  return RopeArgs{r.inv_freq, r.positions, r.rotary_dim / 2, r.rot_start, r.layout, r.mscale,
                  r.backward ? -1.f : 1.f};
}
}  // namespace

// The table of TT tokens in LDS, then every (token, head) in units of V
// elements (V = 16 bytes' worth, or 1 where sizes or alignment do not divide):
// a unit of the rotary part is V pairs' elements (two pieces of V for the half
// layout, one for the interleaved, with pairs inside it; two single elements
// when V = 1), any other unit a copy.  In place, copies are skipped.
template <int DT, int V>
__global__ void __launch_bounds__(kThreads) k_rope(const typename Elem<DT>::T* x, int64_t x_st, int64_t x_sh,
                                                   typename Elem<DT>::T* out, int64_t o_st, int64_t o_sh,
                                                   int64_t n_tokens, int H, int D, int TT, int in_place, RopeArgs r) {
  using E = Elem<DT>;
  using T = typename E::T;
  extern __shared__ float2 s_cs[];   // [TT][half]
  struct alignas(V * sizeof(T)) Vec { T v[V]; };
  const bool split = r.layout == MISA_ROPE_HALF || V == 1;   // a unit's two sides are apart
  const int rot_units = split ? r.half / V : 2 * r.half / V;
  const int pre = r.start / V;                               // copied units before the rotary part
  const int units = rot_units + (in_place ? 0 : (D - 2 * r.half) / V);
  for (int64_t t0 = (int64_t)blockIdx.x * TT; t0 < n_tokens; t0 += (int64_t)gridDim.x * TT) {
    const int nt = (int)min((int64_t)TT, n_tokens - t0);
    for (int i = threadIdx.x; i < nt * r.half; i += kThreads) {
      const int t = i / r.half, j = i - t * r.half;
      const double turns = (double)r.positions[t0 + t] * (r.inv_freq[j] * kInv2Pi);
      if constexpr (DT == MISA_T_FP32) {
        const double2 cs = turn_f64(turns, r.mscale);
        s_cs[i] = make_float2((float)cs.x, (float)cs.y);
      } else {
        s_cs[i] = turn_f32(turns, r.mscale);
      }
    }
    __syncthreads();
    const int total = nt * H * units;
    for (int i = threadIdx.x; i < total; i += kThreads) {
      const int row = i / units, u = i - row * units;
      const int t = row / H, h = row - t * H;
      const T* xr = x + (t0 + t) * x_st + h * x_sh;
      T* orow = out + (t0 + t) * o_st + h * o_sh;
      const float2* cs = s_cs + t * r.half;
      if (u < rot_units) {
        if (split) {
          const int j = u * V;
          const int ia = r.layout == MISA_ROPE_HALF ? r.start + j : r.start + 2 * j;
          const int ib = r.layout == MISA_ROPE_HALF ? ia + r.half : ia + 1;
          const Vec a = *reinterpret_cast<const Vec*>(xr + ia), b = *reinterpret_cast<const Vec*>(xr + ib);
          Vec ya, yb;
  #pragma unroll
          for (int e = 0; e < V; ++e) {
            const float c = cs[j + e].x, s = cs[j + e].y * r.sign, fa = E::load(a.v[e]), fb = E::load(b.v[e]);
            ya.v[e] = E::store(__builtin_fmaf(fa, c, -(fb * s)));
            yb.v[e] = E::store(__builtin_fmaf(fa, s, fb * c));
          }
          *reinterpret_cast<Vec*>(orow + ia) = ya;
          *reinterpret_cast<Vec*>(orow + ib) = yb;
        } else {
          const int at = r.start + u * V;
          const Vec a = *reinterpret_cast<const Vec*>(xr + at);
          Vec y;
  #pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const float2 k = cs[u * (V / 2) + e];
            const float c = k.x, s = k.y * r.sign, fa = E::load(a.v[2 * e]), fb = E::load(a.v[2 * e + 1]);
            y.v[2 * e] = E::store(__builtin_fmaf(fa, c, -(fb * s)));
            y.v[2 * e + 1] = E::store(__builtin_fmaf(fa, s, fb * c));
          }
          *reinterpret_cast<Vec*>(orow + at) = y;
        }
      } else {
        const int w = u - rot_units;
        const int at = (w < pre ? w : w + 2 * r.half / V) * V;
        *reinterpret_cast<Vec*>(orow + at) = *reinterpret_cast<const Vec*>(xr + at);
      }
    }
    __syncthreads();   // the table is free for the next tokens
  }
}

namespace {
template <int DT>
hipError_t rope_type(const RopeArgs& r, const void* x, int64_t x_st, int64_t x_sh, void* out, int64_t o_st,
                     int64_t o_sh, int64_t n, int H, int D, hipStream_t st) {
  using T = typename Elem<DT>::T;
  constexpr int V = 16 / (int)sizeof(T);
  const bool in_place = x == out;
  const int side = r.layout == MISA_ROPE_HALF ? r.half : 2 * r.half;
  const bool vec = side % V == 0 && r.start % V == 0 && D % V == 0 && x_st % V == 0 && x_sh % V == 0 &&
                   o_st % V == 0 && o_sh % V == 0 && ((uintptr_t)x & 15) == 0 && ((uintptr_t)out & 15) == 0;
  // tokens of a workgroup: about 4 units a thread, but no fewer than four
  // workgroups to a CU where the call has them, and a table within 32 KB
  const int units = (D - (in_place ? D - 2 * r.half : 0)) / (vec ? V : 1);
  int64_t TT = std::max<int64_t>(1, 4 * kThreads / std::max<int64_t>(1, (int64_t)H * units));
  TT = std::min<int64_t>(TT, std::max<int64_t>(1, n / 1024));
  TT = std::min<int64_t>(TT, std::max<int64_t>(1, 32768 / (r.half * (int64_t)sizeof(float2))));
  const dim3 grid((unsigned)std::min<int64_t>((n + TT - 1) / TT, kMaxGroups));
  const size_t lds = (size_t)TT * r.half * sizeof(float2);
  if (vec)
    hipLaunchKernelGGL((k_rope<DT, V>), grid, dim3(kThreads), lds, st, static_cast<const T*>(x), x_st, x_sh,
                       static_cast<T*>(out), o_st, o_sh, n, H, D, (int)TT, (int)in_place, r);
  else
    hipLaunchKernelGGL((k_rope<DT, 1>), grid, dim3(kThreads), lds, st, static_cast<const T*>(x), x_st, x_sh,
                       static_cast<T*>(out), o_st, o_sh, n, H, D, (int)TT, (int)in_place, r);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_rope(const misa_rope_spec& spec, const void* x, int dtype, int64_t n_tokens, int H, int D,
                       int64_t x_st, int64_t x_sh, void* out, int64_t o_st, int64_t o_sh, hipStream_t st) {
  const RopeArgs r = rope_args(spec);
  if (dtype == MISA_T_BF16) return rope_type<MISA_T_BF16>(r, x, x_st, x_sh, out, o_st, o_sh, n_tokens, H, D, st);
  if (dtype == MISA_T_FP16) return rope_type<MISA_T_FP16>(r, x, x_st, x_sh, out, o_st, o_sh, n_tokens, H, D, st);
  return rope_type<MISA_T_FP32>(r, x, x_st, x_sh, out, o_st, o_sh, n_tokens, H, D, st);
}

// One row (token, head, k or v) to LPR lanes (LPR = D / 8 rounded up to a power
// of two), 8 values a lane; a pair's other value lies in the lane's own piece
// (interleaved) or in one other piece (half layout), or anywhere (odd offsets).
// Rows that become codes are rotated in fp64: a value that lands on the other
// side of an e4m3 border is an error of half a step, so the value that meets
// the border should be the true one.  Such a value is kept as fp32 x + dx; the
// quotients by which it becomes a scale or a code are those of x, corrected by
// their remainders, and so rounded to fp32 once.
template <bool FP8>
struct Turn {
  using T = double;
  static __device__ __forceinline__ double2 of(double turns, double m) { return turn_f64(turns, m); }
};
template <>
struct Turn<false> {
  using T = float;
  static __device__ __forceinline__ float2 of(double turns, double m) { return turn_f32(turns, m); }
};

__device__ __forceinline__ void unpack8(uint4 w4, float* x) {
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    x[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
  }
}

// A thread keeps its head and side (k or v) and steps through tokens: the
// divisions are done once, and a row's addresses are a product each.
struct WriteArgs {
  const uint16_t *k, *v;   // v nullable
  int64_t k_st, k_sh, v_st, v_sh;
  const int64_t* slots;
  int64_t n_tokens, n_slots;
  int H, D, lpr_log2, TT;
  void *k_pages, *v_pages;
  float *k_scale, *v_scale;
};

// How the keys turn: not at all; whole pieces, half layout (all 8 values of a
// piece on one side, their partners in one other piece); whole pieces,
// interleaved (partners side by side); any other offsets.
enum { kStill = 0, kHalf = 1, kPairs = 2, kAny = 3 };

template <bool FP8, int KIND>
__global__ void __launch_bounds__(kThreads) k_write_pages(const WriteArgs a, const RopeArgs r) {
  using Tn = Turn<FP8>;
  using T = typename Tn::T;
  extern __shared__ double s_raw[];
  T* const s_c = reinterpret_cast<T*>(s_raw);   // [TT][half] cosines, then sines
  T* const s_s = s_c + a.TT * r.half;
  const int lpr = 1 << a.lpr_log2, p = threadIdx.x & (lpr - 1), e0 = p * 8;
  const int grp = threadIdx.x >> a.lpr_log2, groups = kThreads >> a.lpr_log2;
  // a token's rows over the groups of lanes: several tokens to a pass, or several passes to a token
  const int rpt = a.H * (a.v != nullptr ? 2 : 1);
  const int tpp = max(1, groups / rpt), chunks = (rpt + groups - 1) / groups;
  const int sub = chunks == 1 ? grp / rpt : 0, hs0 = chunks == 1 ? grp - sub * rpt : grp;
  const bool live = e0 < a.D;
  const bool hl = r.layout == MISA_ROPE_HALF;
  const int q0 = e0 - r.start;   // first value's place in the rotary part
  const bool turns = KIND != kStill && live && q0 + 8 > 0 && q0 < 2 * r.half;   // (of k rows)
  const bool second0 = q0 >= r.half;
  struct Row {
    uint4 mine, other;
    int64_t slot;
    const uint16_t* src;
    int t, h;
    bool is_v;
  };
  for (int64_t t0 = (int64_t)blockIdx.x * a.TT; t0 < a.n_tokens; t0 += (int64_t)gridDim.x * a.TT) {
    const int nt = (int)min((int64_t)a.TT, a.n_tokens - t0);
    const int items = (nt + tpp - 1) / tpp * chunks;
    auto fetch = [&](int it) __attribute__((always_inline)) -> Row {
      Row w;
      const int pass = chunks == 1 ? it : it / chunks;
      const int hs = chunks == 1 ? hs0 : hs0 + (it - pass * chunks) * groups;
      const int t = pass * tpp + sub;
      const bool in = it < items && sub < tpp && t < nt && hs < rpt;
      w.t = min(t, nt - 1);
      const int hc = min(hs, rpt - 1);
      w.is_v = hc >= a.H;
      w.h = w.is_v ? hc - a.H : hc;
      const int64_t slot = a.slots[t0 + w.t];
      w.slot = in ? slot : -1;
      w.src = w.is_v ? a.v + (t0 + w.t) * a.v_st + w.h * a.v_sh : a.k + (t0 + w.t) * a.k_st + w.h * a.k_sh;
      w.mine = live ? *reinterpret_cast<const uint4*>(w.src + e0) : make_uint4(0, 0, 0, 0);
      w.other = w.mine;
      if (KIND == kHalf && turns && !w.is_v)
        w.other = *reinterpret_cast<const uint4*>(w.src + (second0 ? e0 - r.half : e0 + r.half));
      return w;
    };
    // the first row's loads are under way while the table is formed (two or four
    // rows' cost more in registers, and so in waves, than they gain)
    Row w = fetch(0);
    if (KIND != kStill) {
      for (int i = threadIdx.x; i < nt * r.half; i += kThreads) {
        const int t = i / r.half, j = i - t * r.half;
        const auto cs = Tn::of((double)r.positions[t0 + t] * (r.inv_freq[j] * kInv2Pi), r.mscale);
        s_c[i] = cs.x;
        s_s[i] = cs.y;
      }
      __syncthreads();
    }
    for (int it = 0; it < items; ++it) {
      if (it > 0) w = fetch(it);
      if (w.slot < 0 || w.slot >= a.n_slots) continue;   // uniform over a row's lanes
      float x[8], dx[8] = {};
      unpack8(w.mine, x);
      auto put = [&](int i, T z) __attribute__((always_inline)) {
        x[i] = (float)z;
        if constexpr (FP8) dx[i] = __builtin_fabsf(x[i]) < INFINITY ? (float)(z - (T)x[i]) : 0.f;
      };
      if (turns && !w.is_v) {
        const T *c = s_c + w.t * r.half, *s = s_s + w.t * r.half;
        if constexpr (KIND == kHalf) {
          const int j0 = second0 ? q0 - r.half : q0;
          float y[8];
          unpack8(w.other, y);
#pragma unroll
          for (int i = 0; i < 8; ++i)   // first: a c - b s; second: b c + a s
            put(i, (T)x[i] * c[j0 + i] + (T)(second0 ? y[i] : -y[i]) * s[j0 + i]);
        } else if constexpr (KIND == kPairs) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const int q = q0 + i;
            if (q < 0 || q >= 2 * r.half) continue;
            const T a0 = x[i], b0 = x[i + 1], cj = c[q >> 1], sj = s[q >> 1];
            put(i, a0 * cj - b0 * sj);
            put(i + 1, b0 * cj + a0 * sj);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int q = q0 + i;
            if (q < 0 || q >= 2 * r.half) continue;
            const bool second = hl ? q >= r.half : (q & 1);
            const int j = hl ? (second ? q - r.half : q) : q >> 1;
            const int other = hl ? (second ? q - r.half : q + r.half) : q ^ 1;
            const T mine = x[i], his = bf16_bits_to_f32(w.src[r.start + other]);
            put(i, mine * c[j] + (second ? his : -his) * s[j]);
          }
        }
      }
      const int64_t dst_row = w.slot * a.H + w.h;
      if constexpr (FP8) {
        float sc;
        if constexpr (KIND == kStill) {
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, __builtin_fabsf(x[i]));
          for (int o = lpr >> 1; o >= 1; o >>= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o, lpr));
          sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
        } else {
          double amax = 0.;
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = __builtin_fmax(amax, __builtin_fabs((double)x[i] + (double)dx[i]));
          for (int o = lpr >> 1; o >= 1; o >>= 1) amax = __builtin_fmax(amax, __shfl_xor(amax, o, lpr));
          const float top = (float)amax, rest = (float)(amax - (double)top);
          sc = __fdiv_rn(top, 448.f);
          if (rest != 0.f && top < INFINITY) sc += (__builtin_fmaf(-sc, 448.f, top) + rest) * (1.f / 448.f);
          if (!(amax > 0.)) sc = 1.f;
        }
        float q[8];
        const float inv = KIND == kStill ? 0.f : __fdiv_rn(1.f, sc);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          q[i] = __fdiv_rn(x[i], sc);
          if (KIND != kStill && dx[i] != 0.f && sc < INFINITY) q[i] += (__builtin_fmaf(-q[i], sc, x[i]) + dx[i]) * inv;
        }
        uint32_t c[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          int u = 0;
          u = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], u, false);
          u = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], u, true);
          c[i] = (uint32_t)u;
        }
        uint8_t* pool = static_cast<uint8_t*>(w.is_v ? a.v_pages : a.k_pages);
        if (live) *reinterpret_cast<uint2*>(pool + dst_row * a.D + e0) = make_uint2(c[0], c[1]);
        if (p == 0) (w.is_v ? a.v_scale : a.k_scale)[dst_row] = sc;
      } else {
        uint16_t* pool = static_cast<uint16_t*>(w.is_v ? a.v_pages : a.k_pages);
        if (live)
          *reinterpret_cast<uint4*>(pool + dst_row * a.D + e0) =
              make_uint4(pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7]));
      }
    }
    if (KIND != kStill) __syncthreads();   // the table is free for the next tokens
  }
}

hipError_t launch_write_pages(int64_t n_tokens, int H, int D, const uint16_t* k, int64_t k_st, int64_t k_sh,
                              const uint16_t* v, int64_t v_st, int64_t v_sh, const int64_t* slots,
                              const misa_rope_spec* spec, void* k_pages, void* v_pages, int kdtype, float* k_scale,
                              float* v_scale, int64_t n_slots, hipStream_t st) {
  RopeArgs r{};
  if (spec != nullptr) r = rope_args(*spec);
  int lpr_log2 = 0;
  while ((8 << lpr_log2) < D) ++lpr_log2;
  // tokens of a workgroup: a row for every group of lanes, up to four where that
  // leaves four workgroups to a CU; table within 32 KB
  const int64_t lanes = ((int64_t)H * (v != nullptr ? 2 : 1)) << lpr_log2;
  const int64_t cs_bytes = 2 * (kdtype == MISA_K_FP8_E4M3 ? sizeof(double) : sizeof(float));
  int64_t TT = std::max<int64_t>(1, kThreads / lanes);
  TT = std::max<int64_t>(TT, std::min<int64_t>(4 * kThreads / lanes, n_tokens / 1024));
  if (r.half > 0) TT = std::min<int64_t>(TT, std::max<int64_t>(1, 32768 / (r.half * cs_bytes)));
  const dim3 grid((unsigned)std::min<int64_t>((n_tokens + TT - 1) / TT, kMaxGroups));
  const size_t lds = (size_t)TT * r.half * cs_bytes;
  const WriteArgs a{k, v, k_st, k_sh, v_st, v_sh, slots, n_tokens, n_slots, H, D, lpr_log2, (int)TT,
                    k_pages, v_pages, k_scale, v_scale};
  const int kind = r.half == 0 ? kStill
                   : r.layout == MISA_ROPE_HALF ? (r.start % 8 == 0 && r.half % 8 == 0 ? kHalf : kAny)
                                                : (r.start % 2 == 0 ? kPairs : kAny);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), lds, st, a, r); };
  if (kdtype == MISA_K_FP8_E4M3) {
    if (kind == kStill) go(k_write_pages<true, kStill>);
    else if (kind == kHalf) go(k_write_pages<true, kHalf>);
    else if (kind == kPairs) go(k_write_pages<true, kPairs>);
    else go(k_write_pages<true, kAny>);
  } else {
    if (kind == kStill) go(k_write_pages<false, kStill>);
    else if (kind == kHalf) go(k_write_pages<false, kHalf>);
    else if (kind == kPairs) go(k_write_pages<false, kPairs>);
    else go(k_write_pages<false, kAny>);
  }
  return hipGetLastError();
}

}  // namespace misa
