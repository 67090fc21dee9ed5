// Block tables, slots and packing of a step from the requests' lengths.
//
// With c_b cached and n_b new tokens, page size ps and H(x) = ceil(x / ps),
// request b lacks H(c_b + n_b) - H(c_b) pages. Exclusive prefix sums over the
// requests give its first packed row (cu) and its first taken page, so every
// packed token and every taken page can be placed on its own: token t finds its
// request in cu by bisection, its position is c_b + t - cu_b, and its page is a
// table entry (held before) or an entry of the free stack (taken now).
//
// What bounds it: the chain launch, lengths, scan, bisection, page number, store; the
// bytes (8 per token) are few. So every CTA scans all lengths by itself (at most 4096,
// 8 per thread) in place of a scan kernel. A small plan is one launch of one CTA. A
// large one is two: many CTAs place tokens and pages, then one CTA writes what may lie
// over the inputs (lengths, free count, returned pages), which the first has read by
// then. One CTA places 2048 tokens in about 1.7 us; with 117 thousand tokens of 1000
// requests a cluster of 8 CTAs in one launch takes 17.6 us, 9.6 us this way.
#include "kernels.cuh"

#include <algorithm>

namespace llama {

namespace {
constexpr int PPT = 512;        // threads per CTA
constexpr int PP_MAX_CTAS = 148;
constexpr int PP_PLACE = 1, PP_FINISH = 2;  // parts of a plan
constexpr int PP_WARPS = PPT / 32;
}  // namespace

// last index i in [0, n) with a[i] <= x (a ascending, a[0] <= x)
__device__ __forceinline__ int pp_find(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(PPT) page_plan_kernel(const PagePlanParams p, int parts) {
  extern __shared__ int pp_smem[];
  const int B = p.B;
  int* s_cu = pp_smem;          // [B + 1] packed rows
  int* s_pp = s_cu + B + 1;     // [B + 1] taken pages
  int* s_rp = s_pp + B + 1;     // [B + 1] returned pages
  int* s_c = s_rp + B + 1;      // [B] cached tokens
  __shared__ long long s_w[3][PP_WARPS];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ranks = gridDim.x;
  const int ps1 = (1 << p.page_shift) - 1;
  const int fc = *p.free_count;
  const int per = (B + PPT - 1) / PPT;

  int err = fc < 0 || fc > p.num_pages ? LLAMA_DEV_OUT_OF_PAGES : 0;
  // this thread's requests [b0, b1): sums, then exclusive prefixes
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long sum[3] = {0, 0, 0};
  for (int pass = 0; pass < 2; ++pass) {
    long long at[3];
    if (pass == 1) {
      // exclusive scan of the threads' sums
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        long long x = sum[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (lane == 31) s_w[i][warp] = x;
        at[i] = x - sum[i];
      }
      __syncthreads();
      long long total[3] = {0, 0, 0};
#pragma unroll
      for (int i = 0; i < 3; ++i)
        for (int w = 0; w < PP_WARPS; ++w) {
          if (w < warp) at[i] += s_w[i][w];
          total[i] += s_w[i][w];
        }
      if (total[0] > p.max_tokens) err |= LLAMA_DEV_POS_RANGE;
      if (total[1] > fc || fc - total[1] + total[2] > p.num_pages) err |= LLAMA_DEV_OUT_OF_PAGES;
    }
    for (int b = b0; b < b1; ++b) {
      const int c = p.cached[b], n = p.fresh[b];
      const bool bad = c < 0 || (long long)c + max(n, 0) > ((long long)p.max_pages << p.page_shift);
      if (bad) err |= LLAMA_DEV_POS_RANGE;
      const int held = bad ? 0 : (c + ps1) >> p.page_shift;
      const int tok = bad || n < 0 ? 0 : n;
      const int need = bad || n < 0 ? 0 : ((c + n + ps1) >> p.page_shift) - held;
      const int back = bad || n >= 0 ? 0 : held;
      if (pass == 0) {
        sum[0] += tok;
        sum[1] += need;
        sum[2] += back;
      } else {
        // on a refused plan the sums may not fit; nothing reads them then
        s_cu[b] = (int)at[0];
        s_pp[b] = (int)at[1];
        s_rp[b] = (int)at[2];
        s_c[b] = c;
        at[0] += tok;
        at[1] += need;
        at[2] += back;
        if (b == B - 1) {
          s_cu[B] = (int)at[0];
          s_pp[B] = (int)at[1];
          s_rp[B] = (int)at[2];
        }
      }
    }
  }
  // err of every thread (the flags are few: three votes)
  int all = 0;
  if (__syncthreads_or(err & LLAMA_DEV_POS_RANGE)) all |= LLAMA_DEV_POS_RANGE;
  if (__syncthreads_or(err & LLAMA_DEV_OUT_OF_PAGES)) all |= LLAMA_DEV_OUT_OF_PAGES;
  const bool refused = all != 0;
  const int tokens = refused ? 0 : s_cu[B], taken = refused ? 0 : s_pp[B], returned = refused ? 0 : s_rp[B];
  int flag = all;

  if (parts & PP_PLACE) {
    // packed tokens, four per thread and turn
    for (long long t0 = 4LL * (rank * PPT + tid); t0 < p.max_tokens; t0 += 4LL * PPT * ranks) {
      int pos[4], slot[4];
      int b = t0 < tokens ? pp_find(s_cu, B, (int)t0) : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = (int)min(t0 + i, 0x7fffffffLL);
        pos[i] = 0;
        slot[i] = -1;
        if (t < tokens) {
          while (t >= s_cu[b + 1]) ++b;
          const int c = s_c[b], held = (c + ps1) >> p.page_shift;
          pos[i] = c + t - s_cu[b];
          const int k = pos[i] >> p.page_shift;
          const int page = k < held ? p.tables[(size_t)b * p.max_pages + k] : p.free_pages[fc - 1 - (s_pp[b] + k - held)];
          if ((unsigned)page < (unsigned)p.num_pages)
            slot[i] = (page << p.page_shift) + (pos[i] & ps1);
          else
            flag |= LLAMA_DEV_PAGE_RANGE;
        }
      }
      if (t0 + 3 < p.max_tokens) {
        *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t0 + i < p.max_tokens) {
            p.positions[t0 + i] = pos[i];
            p.slots[t0 + i] = slot[i];
          }
      }
    }
    // taken pages -> the tables' new entries
    for (int e = rank * PPT + tid; e < taken; e += PPT * ranks) {
      const int b = pp_find(s_pp, B, e);
      const int held = (s_c[b] + ps1) >> p.page_shift;
      const int page = p.free_pages[fc - 1 - e];
      if ((unsigned)page >= (unsigned)p.num_pages) flag |= LLAMA_DEV_PAGE_RANGE;
      p.tables[(size_t)b * p.max_pages + held + e - s_pp[b]] = page;
    }
  }
  if (parts & PP_FINISH) {  // by one CTA
    // lengths out: read everything first (kv_lens may be cached_lens)
    __syncthreads();
    for (int b = rank * PPT + tid; b < B; b += PPT * ranks) {
      p.cu[b] = refused ? 0 : s_cu[b];
      p.kv_lens[b] = refused ? s_c[b] : s_rp[b + 1] > s_rp[b] ? 0 : s_c[b] + s_cu[b + 1] - s_cu[b];
    }
    // ended requests' pages go on top of what was left
    for (int e = rank * PPT + tid; e < returned; e += PPT * ranks) {
      const int b = pp_find(s_rp, B, e);
      int page = p.tables[(size_t)b * p.max_pages + e - s_rp[b]];
      if ((unsigned)page >= (unsigned)p.num_pages) {
        flag |= LLAMA_DEV_PAGE_RANGE;
        page = -1;
      }
      p.free_pages[fc - taken + e] = page;
    }
    if (rank == 0 && tid == 0) {
      p.cu[B] = tokens;
      *p.free_count_out = fc - taken + returned;
    }
  }
  if (flag && (rank == 0 || flag != all)) atomicOr(p.status, flag);
}

cudaError_t launch_page_plan(const PagePlanParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  const size_t smem_max = (4 * (size_t)LLAMA_MAX_SEQS + 3) * sizeof(int);
  cudaError_t e = ensure_smem(page_plan_kernel, smem_max, attr);
  if (e != cudaSuccess) return e;
  const size_t smem = (4 * (size_t)p.B + 3) * sizeof(int);
  const int turns = (int)((p.max_tokens + 4LL * PPT - 1) / (4 * PPT));
  if (turns <= 2) {
    page_plan_kernel<<<1, PPT, smem, st>>>(p, PP_PLACE | PP_FINISH);
  } else {
    page_plan_kernel<<<std::min(turns, PP_MAX_CTAS), PPT, smem, st>>>(p, PP_PLACE);
    page_plan_kernel<<<1, PPT, smem, st>>>(p, PP_FINISH);
  }
  return cudaGetLastError();
}

}  // namespace llama
