// Block tables and slot maps from request lengths (misa_plan_pages).
//
// Everything follows from two exclusive sums over the sequences: the new
// tokens (q_start) and the new pages (the offset into the free list).  One
// launch does it all: every workgroup forms both sums for itself (n_seq
// lengths are a few KB that the L2 holds), because the alternative, a scan
// launch before the fill, costs a second launch on a call whose whole work is
// shorter than one.
//
// Sums: thread i sums a run of ceil(n_seq / 256) sequences, the 256 run sums
// are scanned by wave shuffles and kept in LDS (s_tok, s_page: first token and
// first page of each run).  A token finds its run by a binary search in LDS (8
// steps) and its sequence by walking the run; with up to 256 sequences a run
// is one sequence and the walk is empty.
// Sums are 64-bit: n_seq lengths of up to 2^31 pass 32 bits.
//
// Bound by the chain lengths -> sums -> search -> free list -> slots, not by bytes:
// 3.7 us for 64 decodes, 9.2 us for 500 prompts of 1..1024 tokens (3.1 MB).
#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

namespace {
constexpr int kThreads = 256;
constexpr int kTokensPerThread = 4;

struct SeqPages {
  int64_t cached, fresh;   // token counts, negative ones taken as 0
  int32_t have, need;      // pages owned, pages to take (both within the table)
};

__device__ __forceinline__ SeqPages seq_pages(const int32_t* cached, const int32_t* fresh, int b, uint32_t P,
                                              int64_t max_pages) {
  SeqPages r;
  r.cached = max(cached[b], 0);
  r.fresh = max(fresh[b], 0);
  // ceil(x / P) of x < 2^32 in 32-bit arithmetic
  const uint32_t c = (uint32_t)r.cached, e = c + (uint32_t)r.fresh;
  const int64_t have = min((int64_t)(c / P + (c % P != 0)), max_pages);
  const int64_t end = min((int64_t)(e / P + (e % P != 0)), max_pages);
  r.have = (int32_t)have;
  r.need = (int32_t)(end - have);
  return r;
}

// last i in [0, 256) with s[i] <= x (s ascending, s[0] = 0 <= x)
__device__ __forceinline__ int run_of(const int64_t* s, int64_t x) {
  int lo = 0;
#pragma unroll
  for (int step = kThreads / 2; step >= 1; step >>= 1)
    if (s[lo + step] <= x) lo += step;
  return lo;
}
}  // namespace

__global__ void __launch_bounds__(kThreads) k_plan_pages(
    int n_seq, const int32_t* __restrict__ cached_lens, const int32_t* __restrict__ new_lens, uint32_t P,
    const int32_t* __restrict__ free_pages, int n_free, int32_t* block_table, int64_t max_pages,
    int32_t* __restrict__ q_start, int32_t* __restrict__ kv_lens, int64_t* __restrict__ slots,
    int32_t* __restrict__ positions, int64_t n_tokens, int32_t* __restrict__ n_taken) {
  __shared__ int64_t s_tok[kThreads], s_page[kThreads];
  __shared__ int64_t s_wave[2][kThreads / kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int run = (n_seq + kThreads - 1) / kThreads;
  const int b0 = min(tid * run, n_seq), b1 = min(b0 + run, n_seq);

  int64_t tok = 0, page = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqPages sp = seq_pages(cached_lens, new_lens, b, P, max_pages);
    tok += sp.fresh;
    page += sp.need;
  }
  int64_t tok_in = tok, page_in = page;   // inclusive over the wave
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t a = __shfl_up(tok_in, o), c = __shfl_up(page_in, o);
    if (lane >= o) {
      tok_in += a;
      page_in += c;
    }
  }
  if (lane == kWave - 1) {
    s_wave[0][wave] = tok_in;
    s_wave[1][wave] = page_in;
  }
  __syncthreads();
  int64_t total_tok = 0, total_page = 0, tok0 = tok_in - tok, page0 = page_in - page;
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) {
    if (w < wave) {
      tok0 += s_wave[0][w];
      page0 += s_wave[1][w];
    }
    total_tok += s_wave[0][w];
    total_page += s_wave[1][w];
  }
  s_tok[tid] = tok0;
  s_page[tid] = page0;
  __syncthreads();

  if (blockIdx.x == 0) {
    int64_t t = tok0;
    for (int b = b0; b < b1; ++b) {
      const int64_t c = max(cached_lens[b], 0), m = max(new_lens[b], 0);
      q_start[b] = (int32_t)min(t, (int64_t)INT32_MAX);
      kv_lens[b] = (int32_t)min(c + m, (int64_t)INT32_MAX);
      t += m;
    }
    if (tid == 0) {
      q_start[n_seq] = (int32_t)min(total_tok, (int64_t)INT32_MAX);
      n_taken[0] = (int32_t)min(total_page, (int64_t)INT32_MAX);
    }
  }

  // the new table entries
  for (int64_t r = (int64_t)blockIdx.x * kThreads + tid; r < total_page; r += (int64_t)gridDim.x * kThreads) {
    const int u = run_of(s_page, r);
    int64_t first = s_page[u];
    for (int b = u * run; b < min((u + 1) * run, n_seq); ++b) {
      const SeqPages sp = seq_pages(cached_lens, new_lens, b, P, max_pages);
      if (r < first + sp.need) {
        block_table[(int64_t)b * max_pages + sp.have + (r - first)] = r < n_free ? free_pages[r] : -1;
        break;
      }
      first += sp.need;
    }
  }

  // the tokens: page ids come from the free list itself (or the row's old
  // entries), never from entries another workgroup may be writing
  const int64_t t0 = (int64_t)blockIdx.x * (kThreads * kTokensPerThread) + tid;
#pragma unroll
  for (int i = 0; i < kTokensPerThread; ++i) {
    const int64_t t = t0 + i * kThreads;
    if (t >= n_tokens) break;
    int64_t slot = -1;
    int32_t pos = -1;
    if (t < total_tok) {
      const int u = run_of(s_tok, t);
      int64_t first = s_tok[u], pfirst = s_page[u];
      for (int b = u * run; b < min((u + 1) * run, n_seq); ++b) {
        const SeqPages sp = seq_pages(cached_lens, new_lens, b, P, max_pages);
        if (t < first + sp.fresh) {
          const uint32_t p = (uint32_t)sp.cached + (uint32_t)(t - first);
          const uint32_t pg = p / P;
          pos = (int32_t)min(p, (uint32_t)INT32_MAX);
          int32_t id = -1;
          if ((int64_t)pg < sp.have) {
            id = block_table[(int64_t)b * max_pages + pg];
          } else if ((int64_t)pg < (int64_t)sp.have + sp.need) {
            const int64_t r = pfirst + pg - sp.have;
            id = r < n_free ? free_pages[r] : -1;
          }
          if (id >= 0) slot = (int64_t)id * P + (p - pg * P);
          break;
        }
        first += sp.fresh;
        pfirst += sp.need;
      }
    }
    slots[t] = slot;
    positions[t] = pos;
  }
}

hipError_t launch_plan_pages(int n_seq, const int32_t* cached_lens, const int32_t* new_lens, int page_keys,
                             const int32_t* free_pages, int n_free, int32_t* block_table, int64_t max_pages,
                             int32_t* q_start, int32_t* kv_lens, int64_t* slots, int32_t* positions, int64_t n_tokens,
                             int32_t* n_taken, hipStream_t st) {
  const int64_t per = kThreads * kTokensPerThread;
  const int64_t blocks = n_tokens > 0 ? (n_tokens + per - 1) / per : 1;
  hipLaunchKernelGGL(k_plan_pages, dim3((unsigned)blocks), dim3(kThreads), 0, st, n_seq, cached_lens, new_lens,
                     (uint32_t)page_keys, free_pages, n_free, block_table, max_pages, q_start, kv_lens, slots,
                     positions, n_tokens, n_taken);
  return hipGetLastError();
}

}  // namespace misa
