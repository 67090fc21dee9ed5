// Parts shared by the attention kernels of packed rows: a request's lengths with
// their checks, and the list of key tiles that is cut over the CTAs.
#pragma once

#include <vector>

#include "kernels.cuh"

namespace llama {

// Request b's new tokens and keys, from device memory, with the checks of the
// header: false (and the position range flag) for a request that is skipped.
struct RaggedSeq {
  int q0, n_new, kv;  // first row, new tokens, keys
};
__host__ __device__ __forceinline__ bool ragged_seq(const RaggedAttnParams& p, int b, RaggedSeq& s, bool flag) {
  const int c0 = p.cu[b], c1 = p.cu[b + 1];
  s.q0 = c0;
  bool ok = c0 >= 0 && c1 >= c0 && c1 <= p.N && c1 - c0 <= p.max_new;
  s.n_new = ok ? c1 - c0 : 0;
  s.kv = ok ? s.n_new : 0;
  if (p.tables && ok) {
    s.kv = p.kv_lens[b];
    ok = s.kv >= 0 && s.kv <= (p.max_pages << p.page_shift);
  }
  if (!ok) {
    s.n_new = s.kv = 0;
#ifdef __CUDA_ARCH__
    if (flag) atomicOr(p.status, LLAMA_DEV_POS_RANGE);
#endif
  }
  return ok;
}

// ---- the list of tiles
//
// A unit is a block of query rows of one (request, kv head, group of hpc heads): bq
// consecutive new tokens x hpc heads; it needs the key tiles (KT keys each) up to its
// last position. The units, request by request, kv head by kv head, stand in one list
// that is cut into equal contiguous ranges, one per CTA. A unit takes RT_UNIT entries
// of it for what it costs besides its tiles, and one per tile. Where cutting units would
// gain less than their merge costs, every unit takes one entry and none is cut (w.units).
constexpr int RT_PRE = 128;  // prefix sums kept, at equal distances over the requests
constexpr int RT_UNIT = 1;

// bq and KT are powers of two: no divisions (64-bit ones took most of a small call's start)
__host__ __device__ __forceinline__ int rt_log2(int x) {
#ifdef __CUDA_ARCH__
  return 31 - __clz(x);
#else
  return 31 - __builtin_clz((unsigned)x);
#endif
}
__host__ __device__ __forceinline__ int rt_blocks(int n_new, int bq) { return (n_new + bq - 1) >> rt_log2(bq); }
// q tile t of a request: its key tiles; the sum over the tiles before it (all full)
template <int KT>
__host__ __device__ __forceinline__ int rt_tiles(int c, int n_new, int bq, int t) {
  const long long last = min((long long)(t + 1) * bq, (long long)n_new);
  return (int)((c + last + KT - 1) / KT);
}
__host__ __device__ __forceinline__ long long rt_floor_sum(long long m, int lr) {  // sum of i >> lr over i < m
  const long long q = m >> lr;
  return ((q * (q - 1) / 2) << lr) + q * (m - (q << lr));
}
template <int KT>
__host__ __device__ __forceinline__ long long rt_before(int c, int bq, long long t) {
  if (bq >= KT) {
    const int s = bq >> rt_log2(KT);
    return t * (((long long)c + KT - 1) / KT) + s * (t * (t + 1) / 2);
  }
  // ceil((c + (i + 1) bq) / KT) = floor((e + i) / r) + 1 with e = ceil(c / bq), r = KT / bq
  const int lr = rt_log2(KT) - rt_log2(bq);
  const long long e = ((long long)c + bq - 1) >> rt_log2(bq);
  return t + rt_floor_sum(e + t, lr) - rt_floor_sum(e, lr);
}
template <int KT>
__host__ __device__ __forceinline__ long long rt_total(int c, int n_new, int bq, bool units) {
  if (n_new <= 0) return 0;
  const int nt = rt_blocks(n_new, bq);
  if (units) return nt;
  return rt_before<KT>(c, bq, nt - 1) + rt_tiles<KT>(c, n_new, bq, nt - 1) + (long long)RT_UNIT * nt;
}
// entries of a request before its q tile t
template <int KT>
__host__ __device__ __forceinline__ long long rt_entry(int c, int bq, int t, bool units) {
  return units ? t : rt_before<KT>(c, bq, t) + (long long)RT_UNIT * t;
}
__host__ __device__ __forceinline__ long long rt_begin(long long c, long long W, long long G) { return c * W / G; }
__host__ __device__ __forceinline__ long long rt_own(long long x, long long W, long long G) {
  return ((x + 1) * G - 1) / W;
}

// A CTA's walk over its range [x, end) of the list.
struct RtWalk {
  long long x, end;
  bool units;    // the list's entries are units
  int b, zl, t;  // request, (kv head, head group), q tile
  RaggedSeq s;
  int c, nt;       // keys before the new tokens, q tiles
  long long off;   // entries of the unit before x
  // the current segment: key tiles [j0, j1) of n; key tiles that A and B need
  // (0 where the unit has no rows for B); the unit's first entry
  int j0, j1, n, lim[2];
  long long xs;
};

__host__ __device__ __forceinline__ void rt_load(const RaggedAttnParams& p, int bq, RtWalk& w) {
  ragged_seq(p, w.b, w.s, false);
  w.c = max(w.s.kv - w.s.n_new, 0);
  w.nt = rt_blocks(w.s.n_new, bq);
}
// to entry w.x; pre[i]: entries of one head group of the requests before i * per
template <int KT>
__host__ __device__ __forceinline__ void rt_start(const RaggedAttnParams& p, const long long* pre, int HG, int bq, RtWalk& w) {
  if (w.x >= w.end) return;
  int lo = 0, hi = RT_PRE - 1;  // the last i whose entries begin at or before x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] * HG <= w.x) lo = mid; else hi = mid - 1;
  }
  long long off = w.x - pre[lo] * HG, per = 0;
  for (w.b = lo * ((p.B + RT_PRE - 1) / RT_PRE);; ++w.b) {
    rt_load(p, bq, w);
    per = rt_total<KT>(w.c, w.s.n_new, bq, w.units);
    if (off < per * HG || w.b == p.B - 1) break;
    off -= per * HG;
  }
  w.zl = off < (1LL << 31) && per < (1LL << 31) ? (int)((unsigned)off / (unsigned)per) : (int)(off / per);
  off -= w.zl * per;
  int a = 0, z = w.nt - 1;
  while (a < z) {
    const int mid = (a + z + 1) >> 1;
    if (rt_entry<KT>(w.c, bq, mid, w.units) <= off) a = mid; else z = mid - 1;
  }
  w.t = a;
  w.off = off - rt_entry<KT>(w.c, bq, a, w.units);
}
// the next segment with tiles; false at the end of the range
template <int KT>
__host__ __device__ __forceinline__ bool rt_segment(int bq, RtWalk& w) {
  while (w.x < w.end) {
    w.n = rt_tiles<KT>(w.c, w.s.n_new, bq, w.t);
    const long long take = w.units ? 1 : min(RT_UNIT + w.n - w.off, w.end - w.x);
    w.xs = w.x - w.off;
    w.j0 = w.units ? 0 : (int)max(w.off - RT_UNIT, 0LL);
    w.j1 = w.units ? w.n : (int)max(w.off + take - RT_UNIT, 0LL);
    w.x += take;
    w.off += take;
    if (w.j1 > w.j0) {
      const int bh = bq / 2, left = w.s.n_new - w.t * bq;
      const long long first = (long long)w.c + (long long)w.t * bq + KT - 1;
      w.lim[0] = (int)((first + min(left, bh)) / KT);
      w.lim[1] = left > bh ? (int)((first + min(left, bq)) / KT) : 0;
      return true;
    }
  }
  return false;
}
// on to the next unit, where the segment ended its unit
__host__ __device__ __forceinline__ void rt_advance(const RaggedAttnParams& p, int HG, int bq, RtWalk& w) {
  if (w.x >= w.end) return;
  w.off = 0;
  if (++w.t < w.nt) return;
  w.t = 0;
  if (++w.zl < HG) return;
  w.zl = 0;
  do {
    ++w.b;
    rt_load(p, bq, w);
  } while (w.b < p.B - 1 && w.s.n_new == 0);
}

// Prefix sums of the requests' list entries (one head group), by all threads of a CTA
// (at least RT_PRE); pre[i]: those of the requests before i * ceil(B / RT_PRE).
// Returns whether the entries are units: where the CTA with the most of them takes no
// more tiles than an equal share and MERGE, the merge's cost in tiles. Ends with a
// barrier; s_w: three values per warp of the first RT_PRE threads.
template <int KT, int MERGE>
__device__ __forceinline__ bool rt_prefix(const RaggedAttnParams& p, int bq, int HG, long long* pre, long long* s_w) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int warps = RT_PRE / 32;  // the first RT_PRE threads take them
  const int per = (p.B + RT_PRE - 1) / RT_PRE;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long sum[2] = {0, 0}, most = 0;  // entries by tiles and by units, entries of the longest unit
  RaggedSeq s;
  for (int b = b0; b < b1; ++b) {
    ragged_seq(p, b, s, blockIdx.x == 0);
    if (s.n_new == 0) continue;
    const int c = max(s.kv - s.n_new, 0), nt = rt_blocks(s.n_new, bq);
    sum[0] += rt_total<KT>(c, s.n_new, bq, false);
    sum[1] += nt;
    most = max(most, (long long)RT_UNIT + rt_tiles<KT>(c, s.n_new, bq, nt - 1));
  }
  long long x[2] = {sum[0], sum[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long y = __shfl_up_sync(0xffffffffu, x[i], o);
      if (lane >= o) x[i] += y;
    }
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  if (lane == 31 && warp < warps) {
    s_w[warp] = x[0];
    s_w[warps + warp] = x[1];
    s_w[2 * warps + warp] = most;
  }
  __syncthreads();
  long long total[2] = {0, 0};
  x[0] -= sum[0];
  x[1] -= sum[1];
#pragma unroll
  for (int w = 0; w < warps; ++w) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (w < warp) x[i] += s_w[i * warps + w];
      total[i] += s_w[i * warps + w];
    }
    most = max(most, s_w[2 * warps + w]);
  }
  const long long G = gridDim.x, U = total[1] * HG;
  const bool units = U < (1LL << 30) && (long long)((unsigned)(U + G - 1) / (unsigned)G) * most * G <= total[0] * HG + MERGE * G;
  if (tid < RT_PRE) pre[tid] = units ? x[1] : x[0];
  if (tid == RT_PRE - 1) pre[RT_PRE] = units ? total[1] : total[0];
  __syncthreads();
  return units;
}

// Host walk of the list for lengths in host memory, with the kernels' own functions:
// every key tile of every unit in exactly one CTA's range, in order, and each cut unit
// merged from one partial of each CTA it spans, in the slots the merge reads, no slot or
// counter used twice or outside the workspace. rows: query rows of a unit.
template <int KT>
bool check_ragged_list(const RaggedAttnParams& p, int rows, int grid, bool by_units) {
  const int hpc = prefill_heads_per_cta(p.H / p.Hkv), bq = rows / hpc, HG = p.H / hpc;
  if (rows % hpc || p.H % hpc) return false;
  std::vector<long long> pre(RT_PRE + 1, 0);
  const int per = (p.B + RT_PRE - 1) / RT_PRE;
  long long units = 0;
  for (int b = 0; b < RT_PRE * per; ++b) {
    if (b % per == 0) pre[b / per + 1] = pre[b / per];
    if (b >= p.B) continue;
    RaggedSeq s;
    ragged_seq(p, b, s, false);
    pre[b / per + 1] += rt_total<KT>(s.kv > s.n_new ? s.kv - s.n_new : 0, s.n_new, bq, by_units);
    units += (long long)rt_blocks(s.n_new, bq) * HG;
  }
  const long long W = pre[RT_PRE] * HG, G = W < grid ? W : grid;
  std::vector<char> slot_used(2 * (size_t)grid, 0), counter_used(grid, 0);
  long long done = 0;
  int b = -1, zl = 0, at = 0, from = 0;  // the unit under way, its tiles so far, its first CTA
  int t = 0;
  for (int cta = 0; cta < G; ++cta) {
    RtWalk w;
    w.units = by_units;
    w.x = rt_begin(cta, W, G);
    w.end = rt_begin(cta + 1, W, G);
    const long long xbeg = w.x;
    rt_start<KT>(p, pre.data(), HG, bq, w);
    for (; rt_segment<KT>(bq, w); rt_advance(p, HG, bq, w)) {
      if (w.j0 == 0) {
        if (b >= 0) return false;  // the unit before is not done
        b = w.b, zl = w.zl, t = w.t, at = 0, from = cta;
      }
      const long long c = w.s.kv > w.s.n_new ? w.s.kv - w.s.n_new : 0;
      const long long end = (long long)(w.t + 1) * bq < w.s.n_new ? (long long)(w.t + 1) * bq : w.s.n_new;
      if (b != w.b || zl != w.zl || t != w.t || at != w.j0 || w.n != (c + end + KT - 1) / KT || w.j1 > w.n) return false;
      if (w.zl < 0 || w.zl >= HG || w.t * (long long)bq >= w.s.n_new) return false;
      at = w.j1;
      const bool whole = w.j0 == 0 && w.j1 == w.n;
      if (by_units && !whole) return false;
      if (!whole) {
        const long long x0 = w.xs + RT_UNIT;
        const int c0 = (int)rt_own(x0, W, G), c1 = (int)rt_own(x0 + w.n - 1, W, G);
        const int slot = 2 * cta + (w.xs <= xbeg ? 0 : 1);
        if (c0 != from || cta < c0 || cta > c1 || (w.j1 == w.n) != (cta == c1)) return false;
        if (slot != (cta == c0 ? 2 * c0 + (w.xs <= rt_begin(c0, W, G) ? 0 : 1) : 2 * cta) || slot_used[slot]) return false;
        slot_used[slot] = 1;
        if (cta == c0 && counter_used[c0]) return false;
        counter_used[c0] = 1;
      }
      if (w.j1 == w.n) {
        b = -1;
        ++done;
      }
    }
  }
  return b < 0 && done == units;
}

// packed fp32 arithmetic: two lanes of a 64-bit register per instruction
__device__ __forceinline__ uint64_t rt_f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void rt_split(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t rt_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t rt_mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t rt_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// One thread of the warp, as elect.sync names it: the compiler then knows that code under
// it runs in one thread, and issues tcgen05 instructions without a loop over lanes (8
// MMAs in 122 cycles against 423 under a test of the lane number, a commit in 5
// against 45).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

}  // namespace llama
