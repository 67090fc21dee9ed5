// Causal attention of packed rows on the 5th-generation tensor cores, over a
// paged cache or over packed keys (bf16): chunks of new tokens, whole prompts,
// and batches that mix them with single tokens.
//
// For the i-th of the n new tokens of a request with kv keys, position
// p = kv - n + i, and query head h: softmax_j(q.k_j / sqrt(D)) over the keys
// j <= p of kv head h / n_rep, times V.
//
// A unit is 256 query rows of one (request, kv head): hpc query heads (the
// largest power of two up to 8 dividing n_rep) x 256 / hpc positions, as two
// tiles A and B of 128 rows. It walks the 128-key tiles up to its last
// position. The tiles of all units, unit-major, form one list that is cut into
// equal contiguous ranges, one per CTA and one CTA per SM, so the CTAs finish
// together whatever the lengths; a unit cut between CTAs leaves unnormalised
// partials (max, sum, O), merged in CTA order by the CTA that arrives last.
//   warp 0      TMA: Q (two boxes of 128 rows), then K(j), V(j) in turn through
//               a ring of 128-key stages (128-byte swizzle, no multicast); a
//               stage is 128 / page_size page boxes, a lane each. Pages past
//               the request's last one are read as out of range, i.e. zeros;
//   warp 1      one thread issues the MMAs: for each key tile, for A then B:
//               O += P V (P from TMEM, where the softmax wrote it over S), then
//               the next S = Q K^T. MMAs of one thread run in order, so S may
//               overwrite the P that the MMA before it reads, and the commit
//               behind S also tells the softmax that O is at rest;
//   warps 4..7  softmax of tile A, one thread per row (its TMEM lane);
//   warps 8..11 softmax of tile B. While one tile's softmax runs, the tensor
//               core works on the other's.
// A thread raises its running maximum only when a score passes it by more than
// 2^8 (O and the sum are then rescaled), so P <= 2^8.
//
// P is rounded to one bf16 for the product with V (fp32 sum of the unrounded
// values): a second part of the remainder would raise the MMA work by half and
// take the error from 1.4 to 1.0 times that of rounding the output alone.
//
// V rows past the request's last key hold whatever the page or the next prompt
// holds; 0 x NaN is NaN in the MMA, so the softmax threads zero those rows of
// the last tile in shared memory before they hand over P. A V row that is not
// finite inside the diagonal tile would reach the earlier rows of its tile the
// same way: rows whose result is not finite are computed again, key by key.
#include <algorithm>

#include "ragged.cuh"

namespace llama {

namespace {
constexpr int RT_KT = 128;  // keys per tile
constexpr int RT_THREADS = 384;
constexpr int RT_LEADER = 128;  // first softmax thread
constexpr float RT_LOG2E = 1.4426950408889634f;
constexpr float RT_RESCALE = 8.0f;  // raise the running maximum only past 2^8
}  // namespace

template <int D>
struct RtCfg {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t HALF = RT_KT * 128;          // 128 rows x 64 bf16
  static constexpr uint32_t TILE = HALVES * HALF;        // a Q tile or a K or V stage
  static constexpr int STAGES = 131072 / TILE;           // 128 KB of ring
  static constexpr uint32_t S_COL = 0, O_COL = 256;      // S/P of A, B at 0, 128; O of A, B at 256, 384
  static constexpr int BARS = 2 * STAGES + 10;
  static constexpr size_t SMEM = 1024 + 2 * TILE + STAGES * TILE + BARS * 8 + 16;
};

// ---- the list of tiles

// q tile t of a request: its key tiles; the sum over the tiles before it (all full)
__host__ __device__ __forceinline__ int rt_tiles(int c, int n_new, int bq, int t) {
  const long long last = min((long long)(t + 1) * bq, (long long)n_new);
  return (int)((c + last + RT_KT - 1) / RT_KT);
}
__host__ __device__ __forceinline__ long long rt_floor_sum(long long m, int r) {  // sum of i / r over i < m
  const long long q = m / r;
  return r * (q * (q - 1) / 2) + q * (m - q * r);
}
__host__ __device__ __forceinline__ long long rt_before(int c, int bq, long long t) {
  if (bq >= RT_KT) {
    const int s = bq / RT_KT;
    return t * (((long long)c + RT_KT - 1) / RT_KT) + s * (t * (t + 1) / 2);
  }
  // ceil((c + (i + 1) bq) / 128) = floor((e + i) / r) + 1 with e = ceil(c / bq), r = 128 / bq
  const int r = RT_KT / bq;
  const long long e = ((long long)c + bq - 1) / bq;
  return t + rt_floor_sum(e + t, r) - rt_floor_sum(e, r);
}
__host__ __device__ __forceinline__ long long rt_total(int c, int n_new, int bq) {
  if (n_new <= 0) return 0;
  const int nt = (n_new + bq - 1) / bq;
  return rt_before(c, bq, nt - 1) + rt_tiles(c, n_new, bq, nt - 1);
}
__host__ __device__ __forceinline__ long long rt_begin(long long c, long long W, long long G) { return c * W / G; }
__host__ __device__ __forceinline__ long long rt_own(long long x, long long W, long long G) { return ((x + 1) * G - 1) / W; }

struct RtUnit {
  int b, zl, t;  // request, (kv head, head group), q tile
  RaggedSeq s;
  int c, nt;     // keys before the new tokens, q tiles
};

__device__ __forceinline__ void rt_load(const RaggedAttnParams& p, int bq, RtUnit& u) {
  ragged_seq(p, u.b, u.s, false);
  u.c = max(u.s.kv - u.s.n_new, 0);
  u.nt = (u.s.n_new + bq - 1) / bq;
}
// pre[b]: tiles of one head group of the requests before b
__device__ __forceinline__ int rt_locate(const RaggedAttnParams& p, const long long* pre, int HG, int bq, long long x,
                                         RtUnit& u) {
  int lo = 0, hi = p.B - 1;  // the last b whose tiles begin at or before x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] * HG <= x) lo = mid; else hi = mid - 1;
  }
  u.b = lo;
  rt_load(p, bq, u);
  const long long per = pre[lo + 1] - pre[lo];
  long long off = x - pre[lo] * HG;
  u.zl = (int)(off / per);
  off -= u.zl * per;
  int a = 0, z = u.nt - 1;
  while (a < z) {
    const int mid = (a + z + 1) >> 1;
    if (rt_before(u.c, bq, mid) <= off) a = mid; else z = mid - 1;
  }
  u.t = a;
  return (int)(off - rt_before(u.c, bq, a));
}
__device__ __forceinline__ void rt_next(const RaggedAttnParams& p, const long long* pre, int HG, int bq, RtUnit& u) {
  if (++u.t < u.nt) return;
  u.t = 0;
  if (++u.zl < HG) return;
  u.zl = 0;
  do ++u.b;
  while (u.b < p.B - 1 && pre[u.b + 1] == pre[u.b]);
  rt_load(p, bq, u);
}

// ---- tensor-core and TMEM forms

__device__ __forceinline__ void rt_mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// 128-byte swizzle, N-major operand: 64-wide column halves lbo apart, 8-row groups 1 KB apart
__device__ __forceinline__ uint64_t rt_desc_n(uint32_t addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFF) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void rt_tma_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void rt_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void rt_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void rt_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void rt_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
__device__ __forceinline__ uint64_t rt_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float rt_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float rt_ex2(float x) {  // 2^x on the special-function unit; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(RT_THREADS, 1)
    attn_ragged_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const RaggedAttnParams p, float* __restrict__ part,
                          int* __restrict__ counters, int hpc) {
  using Cfg = RtCfg<D>;
  constexpr int ST = Cfg::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sKV = sQ + 2 * Cfg::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + ST * Cfg::TILE);
  uint64_t* kv_full = bars;            // [ST] stage i % ST holds the i-th of K(0), V(0), K(1), V(1), ...
  uint64_t* kv_empty = kv_full + ST;   // [ST]
  uint64_t* q_full = kv_empty + ST;    // the segment's Q is in
  uint64_t* q_empty = q_full + 1;      // its last S has finished
  uint64_t* s_full = q_empty + 1;      // [2] S of tile A / B written (and every MMA before it finished)
  uint64_t* p_full = s_full + 2;       // [2] P written over S
  uint64_t* o_full = p_full + 2;       // [2] the segment's last P V has finished
  uint64_t* o_free = o_full + 2;       // [2] O has been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_free + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_last = reinterpret_cast<int*>(tmem_slot + 2);
  long long* pre = reinterpret_cast<long long*>(tmem_slot + 4);  // [B + 1]
  __shared__ long long s_w[RT_THREADS / 32];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_rep = p.H / p.Hkv, groups = n_rep / hpc, HG = p.Hkv * groups;
  const int bq = 256 / hpc, bh = 128 / hpc;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 128);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  {
    // prefix sums of the requests' tiles
    const int per = (p.B + RT_THREADS - 1) / RT_THREADS;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long sum = 0;
    RaggedSeq s;
    for (int b = b0; b < b1; ++b) {
      ragged_seq(p, b, s, blockIdx.x == 0);
      sum += rt_total(max(s.kv - s.n_new, 0), s.n_new, bq);
    }
    long long x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_w[warp] = x;
    __syncthreads();
    x -= sum;
    for (int w = 0; w < warp; ++w) x += s_w[w];
    for (int b = b0; b < b1; ++b) {
      pre[b] = x;
      ragged_seq(p, b, s, false);
      x += rt_total(max(s.kv - s.n_new, 0), s.n_new, bq);
      if (b == p.B - 1) pre[p.B] = x;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long W = pre[p.B] * HG, G = min((long long)gridDim.x, W), cta = blockIdx.x;
  const long long xbeg = cta < G ? rt_begin(cta, W, G) : 0, xend = cta < G ? rt_begin(cta + 1, W, G) : 0;

  // A segment: key tiles [j0, j1) of unit u; tile A has work up to na, B up to nb
  // (0 where the unit has no rows for B)
  RtUnit u;
  int j0 = 0;
  if (xbeg < xend) j0 = rt_locate(p, pre, HG, bq, xbeg, u);
  auto limits = [&](const RtUnit& v, int& na, int& nb) {
    const int left = v.s.n_new - v.t * bq;
    nb = left > bh ? rt_tiles(v.c, v.s.n_new, bq, v.t) : 0;
    na = (int)((v.c + (long long)v.t * bq + min(left, bh) + RT_KT - 1) / RT_KT);
  };

  // 168 registers a thread at launch; the softmax threads hold a row of S and take
  // what the first four warps (two of them idle) give back: 88 + 2 x 208 = 3 x 168
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&map_q);
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_v);
    }
    int i = 0, seg = 0;
    bool ok = true;
    for (long long x = xbeg; ok && x < xend; ++seg) {
      const int n_u = rt_tiles(u.c, u.s.n_new, bq, u.t);
      const int j1 = (int)min((long long)n_u, j0 + (xend - x));
      int na, nb;
      limits(u, na, nb);
      const int kvh = u.zl / groups, h0 = kvh * n_rep + (u.zl - kvh * groups) * hpc;
      if (lane == 0) {
        ok = wait_or_abort(q_empty, (seg & 1) ^ 1, p.status, abort_flag);
        if (ok) {
          mbar_arrive_expect_tx(q_full, (nb ? 2 : 1) * Cfg::TILE);
          for (int g = 0; g < (nb ? 2 : 1); ++g)
#pragma unroll
            for (int hf = 0; hf < Cfg::HALVES; ++hf)
              rt_tma_3d(sQ + g * Cfg::TILE + hf * Cfg::HALF, &map_q, q_full, hf * 64, h0, u.s.q0 + u.t * bq + g * bh);
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0);
      // lane -> (64-wide half, page of the tile); one box per lane
      const int ps = PAGED ? 1 << p.page_shift : RT_KT, boxes = Cfg::HALVES * (RT_KT / ps);
      const int hf = lane % Cfg::HALVES, pg = lane / Cfg::HALVES;
      const int n_pages = PAGED ? (u.s.kv + ps - 1) >> p.page_shift : 0;
      for (int j = j0; ok && j < j1; ++j) {
        int row = 0;
        if (PAGED && lane < boxes) {
          const int k = j * (RT_KT / ps) + pg;
          row = p.num_pages * p.Hkv * ps;  // out of range: zeros
          if (k < n_pages) {
            const int page = __ldg(p.tables + (size_t)u.b * p.max_pages + k);
            if ((unsigned)page < (unsigned)p.num_pages)
              row = (page * p.Hkv + kvh) * ps;
            else
              atomicOr(p.status, LLAMA_DEV_PAGE_RANGE);
          }
        }
#pragma unroll
        for (int kv = 0; kv < 2 && ok; ++kv, ++i) {
          const int st = i % ST;
          ok = wait_or_abort(&kv_empty[st], ((i / ST) & 1) ^ 1, p.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&kv_full[st], Cfg::TILE);
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = sKV + st * Cfg::TILE + hf * Cfg::HALF + pg * ps * 128;
            const CUtensorMap* map = kv ? &map_v : &map_k;
            if (PAGED)
              tma_load_2d(dst, map, &kv_full[st], hf * 64, row);
            else
              rt_tma_3d(dst, map, &kv_full[st], hf * 64, kvh, u.s.q0 + j * RT_KT);
          }
        }
      }
      x += j1 - j0;
      j0 = 0;
      if (x < xend) rt_next(p, pre, HG, bq, u);
    }
    // every copy lands before the CTA can retire
    if (lane == 0) {
      if (seg > 0) mbar_wait(q_full, (seg - 1) & 1, p.status);
      for (int k = (i > ST ? i - ST : 0); k < i; ++k) mbar_wait(&kv_full[k % ST], (k / ST) & 1, p.status);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc_s = make_idesc_bf16(128, RT_KT);
      constexpr uint32_t idesc_pv = make_idesc_bf16(128, D) | (1u << 16);  // B (= V) N-major
      int i = 0, seg = 0;
      int pc[2] = {0, 0};  // P tiles taken of A, B
      int oc[2] = {0, 0};  // segments with work of A, B
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t ph) { return ok = ok && wait_or_abort(bar, ph, p.status, abort_flag); };
      auto issue_s = [&](int g, int slot) {
        const uint32_t qa = smem_u32(sQ + g * Cfg::TILE), ka = smem_u32(sKV + (slot % ST) * Cfg::TILE);
        const uint32_t sd = tmem + Cfg::S_COL + g * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * Cfg::HALF + (kk & 3) * 32;
          tc_mma_bf16(sd, make_sw128_desc(qa + off), make_sw128_desc(ka + off), idesc_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[g]);
      };
      for (long long x = xbeg; ok && x < xend; ++seg) {
        const int n_u = rt_tiles(u.c, u.s.n_new, bq, u.t);
        const int j1 = (int)min((long long)n_u, j0 + (xend - x));
        int lim[2];
        limits(u, lim[0], lim[1]);
        if (!wait(q_full, seg & 1) || !wait(&kv_full[i % ST], (i / ST) & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (j0 < lim[g]) issue_s(g, i);
        tc_commit(&kv_empty[i % ST]);
        if (j1 - j0 == 1) tc_commit(q_empty);
        for (int j = j0; ok && j < j1; ++j, i += 2) {
          const int vs = i + 1, ks = i + 2;  // ring slots of V(j), K(j + 1)
          if (!wait(&kv_full[vs % ST], (vs / ST) & 1)) break;
          if (j + 1 < j1 && !wait(&kv_full[ks % ST], (ks / ST) & 1)) break;
          const uint32_t va = smem_u32(sKV + (vs % ST) * Cfg::TILE);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (j >= lim[g]) continue;
            if (!wait(&p_full[g], pc[g] & 1)) break;
            ++pc[g];
            if (j == j0) {
              if (!wait(&o_free[g], (oc[g] & 1) ^ 1)) break;
              ++oc[g];
            }
            tc_fence_after();
            const uint32_t od = tmem + Cfg::O_COL + g * 128, pa = tmem + Cfg::S_COL + g * 128;
#pragma unroll
            for (int kk = 0; kk < RT_KT / 16; ++kk)
              rt_mma_ts(od, pa + kk * 8, rt_desc_n(va + kk * 2048, Cfg::HALF), idesc_pv, (j > j0 || kk > 0) ? 1u : 0u);
            if (j + 1 < j1 && j + 1 < lim[g])
              issue_s(g, ks);
            else
              tc_commit(&o_full[g]);
          }
          if (!ok) break;
          tc_commit(&kv_empty[vs % ST]);
          if (j + 1 < j1) tc_commit(&kv_empty[ks % ST]);
          if (j + 2 == j1) tc_commit(q_empty);  // the segment's last S has been issued
        }
        x += j1 - j0;
        j0 = 0;
        if (x < xend) rt_next(p, pre, HG, bq, u);
      }
      // every MMA finishes before TMEM is freed: the softmax warps wait for all of
      // them (o_full), except after a timeout
      if (!ok) {
        tc_commit(q_empty);
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < LLAMA_WAIT_LIMIT_NS / 16) {
        }
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // -------------------------------------------------------------------- softmax
    const int g = warp >= 8 ? 1 : 0;
    const int quarter = warp & 3, r = quarter * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_cols = lanes + Cfg::S_COL + g * 128, o_cols = lanes + Cfg::O_COL + g * 128;
    const float sl2 = rsqrtf((float)D) * RT_LOG2E;
    const uint64_t scale2 = rt_f2(sl2, sl2);
    const int pos_l = r / hpc, hl = r - pos_l * hpc;
    const int stride = 256 * D + 512;  // floats of one partial
    int tiles = 0;                     // key tiles walked (ring slots 2 tiles, 2 tiles + 1)
    int sc = 0, oc = 0;                // S tiles taken, segments with work
    bool ok = true;
    for (long long x = xbeg; x < xend;) {
      const int n_u = rt_tiles(u.c, u.s.n_new, bq, u.t);
      const int j1 = (int)min((long long)n_u, j0 + (xend - x));
      int lim[2];
      limits(u, lim[0], lim[1]);
      const int jl = min(j1, lim[g]);  // this tile's rows have work on [j0, jl)
      const int tok = u.t * bq + g * bh + pos_l;
      // last key this row sees (rows past the last token follow it)
      const int last = min(u.s.kv - u.s.n_new + min(tok, u.s.n_new - 1), u.s.kv - 1);
      const bool live = __any_sync(0xffffffffu, tok < u.s.n_new);  // else no row of this warp is anyone's
      float m_used = -INFINITY, l = 0.f;
      for (int j = j0; ok && j < jl; ++j, ++sc) {
        ok = wait_or_abort(&s_full[g], sc & 1, p.status, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int key0 = j * RT_KT;
        if (live) {
        float s[RT_KT];
#pragma unroll
        for (int c = 0; c < 4; ++c) rt_ld32(s_cols + 32 * c, s + 32 * c);
        rt_ld_wait();
        if (__any_sync(0xffffffffu, key0 + RT_KT - 1 > last)) {
#pragma unroll
          for (int c = 0; c < RT_KT; ++c)
            if (key0 + c > last) s[c] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < RT_KT - 4; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = rt_max3(mx[e], s[c + 2 * e], s[c + 2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[RT_KT - 4 + e]);
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;  // log2 units
        if (j == j0) {
          m_used = mt;
        } else if (__any_sync(0xffffffffu, mt > m_used + RT_RESCALE)) {
          // S(j) was issued behind P(j - 1) V(j - 1), so O is at rest
          const float m_new = fmaxf(m_used, mt);
          const float alpha = m_new == -INFINITY ? 1.f : rt_ex2(m_used - m_new);
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float ov[32];
            rt_ld32(o_cols + c, ov);
            rt_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] *= alpha;
            rt_st32(o_cols + c, reinterpret_cast<const uint32_t*>(ov));
          }
          m_used = m_new;
        }
        // p = 2^(s log2(e) / sqrt(D) - m) -> bf16 pairs over this row's S
        const float m_ref = m_used == -INFINITY ? 0.f : m_used;
        const uint64_t negm2 = rt_f2(-m_ref, -m_ref);
        uint64_t ls[2] = {rt_f2(0.f, 0.f), rt_f2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t ph[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float t0, t1;
            rt_split(rt_fma2(rt_f2(s[64 * h + 2 * e], s[64 * h + 2 * e + 1]), scale2, negm2), t0, t1);
            const float p0 = rt_ex2(t0), p1 = rt_ex2(t1);
            ls[e & 1] = rt_add2(ls[e & 1], rt_f2(p0, p1));
            ph[e] = pack_bf16x2(p0, p1);
          }
          rt_st32(s_cols + 32 * h, ph);
        }
        float a0, a1, b0, b1;
        rt_split(ls[0], a0, a1);
        rt_split(ls[1], b0, b1);
        l += (a0 + a1) + (b0 + b1);
        }
        if (key0 + RT_KT > u.s.kv) {
          // V rows past the last key: zeros, before the MMA may read them
          const int vs = 2 * (tiles + j - j0) + 1, row0 = max(u.s.kv - key0, 0);
          ok = wait_or_abort(&kv_full[vs % ST], (vs / ST) & 1, p.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* v = sKV + (vs % ST) * Cfg::TILE;
          const int n16 = (RT_KT - row0) * 8;  // 16-byte pieces of one half
          for (int e = r; e < n16 * Cfg::HALVES; e += 128)
            *reinterpret_cast<uint4*>(v + (e / n16) * Cfg::HALF + row0 * 128 + (e % n16) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        rt_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[g]);
      }
      // after a timeout the warps still walk the segments, for the named barriers below
      if (ok && j0 < jl) {
        ok = wait_or_abort(&o_full[g], oc & 1, p.status, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        ++oc;
        tc_fence_after();
      }
      const bool work = ok && j0 < jl;
      const int kvh = u.zl / groups, h = kvh * n_rep + (u.zl - kvh * groups) * hpc + hl;
      const bool store = ok && tok < u.s.n_new && lim[g] > 0;
      bf16* dst = reinterpret_cast<bf16*>(p.o) + ((size_t)(u.s.q0 + tok) * p.H + h) * D;
      bool bad = false;  // the row's result is not finite
      if (j0 == 0 && j1 == n_u) {
        const float inv = last < 0 ? 0.f : 1.f / l;  // a row without keys is zero
        if (work) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float ov[32];
            rt_ld32(o_cols + c, ov);
            rt_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              ov[e] = last < 0 ? 0.f : ov[e] * inv;
              bad |= !(fabsf(ov[e]) < INFINITY);
            }
            if (store)
#pragma unroll
              for (int e = 0; e < 32; e += 8) store8(dst + c + e, ov + e);
          }
          tc_fence_before();
          mbar_arrive(&o_free[g]);
        }
        bad = bad && store;
      } else {
        // partial: O as [D / 4][256 rows] float4, then (max, sum) per row
        const long long xs = x - j0;  // the unit's first tile
        float* pp = part + (size_t)(2 * cta + (xs <= xbeg ? 0 : 1)) * stride;
        const int row = g * 128 + r;
        if (work) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float ov[32];
            rt_ld32(o_cols + c, ov);
            rt_ld_wait();
            if (store)
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                __stcg(reinterpret_cast<float4*>(pp) + ((c + e) / 4) * 256 + row,
                       make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]));
          }
          tc_fence_before();
          mbar_arrive(&o_free[g]);
        }
        if (store) __stcg(reinterpret_cast<float2*>(pp + 256 * D) + row, make_float2(m_used, l));
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const long long c0 = rt_own(xs, W, G), c1 = rt_own(xs + n_u - 1, W, G);
        if (tid == RT_LEADER) *s_last = ok && atomic_add_acq_rel(&counters[c0], 1) == (int)(c1 - c0);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (*s_last) {
          // partials of CTAs c0 .. c1 in that order; c0 holds the unit in its second
          // slot unless its range starts at the unit, the others in their first
          const long long slot0 = 2 * c0 + (rt_begin(c0, W, G) == xs ? 0 : 1);
          if (store) {
            float mm = -INFINITY;
            for (long long c = c0; c <= c1; ++c)
              mm = fmaxf(mm, __ldcg(reinterpret_cast<const float2*>(part + (c == c0 ? slot0 : 2 * c) * stride + 256 * D) + row).x);
            float ll = 0.f;
            for (long long c = c0; c <= c1; ++c) {
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(part + (c == c0 ? slot0 : 2 * c) * stride + 256 * D) + row);
              if (ml.x != -INFINITY) ll += ml.y * rt_ex2(ml.x - mm);
            }
            const float inv = last < 0 ? 0.f : 1.f / ll;
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
              float acc[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[e] = 0.f;
              for (long long c = c0; c <= c1; ++c) {
                const float* pc = part + (c == c0 ? slot0 : 2 * c) * stride;
                const float m_c = __ldcg(reinterpret_cast<const float2*>(pc + 256 * D) + row).x;
                if (m_c == -INFINITY) continue;  // no weight there (and perhaps no O)
                const float f = rt_ex2(m_c - mm);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const float4 v = __ldcg(reinterpret_cast<const float4*>(pc) + ((d + e) / 4) * 256 + row);
                  acc[e] += v.x * f;
                  acc[e + 1] += v.y * f;
                  acc[e + 2] += v.z * f;
                  acc[e + 3] += v.w * f;
                }
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                acc[e] = last < 0 ? 0.f : acc[e] * inv;
                bad |= !(fabsf(acc[e]) < INFINITY);
              }
              store8(dst + d, acc);
              store8(dst + d + 8, acc + 8);
            }
          }
          if (tid == RT_LEADER) counters[c0] = 0;  // re-armed for the next launch
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");  // s_last is written again by the next split segment
      }
      for (unsigned todo = __ballot_sync(0xffffffffu, bad); todo; todo &= todo - 1) {
        const int src = __ffs(todo) - 1;
        ragged_row<bf16, D>(p, u.b, u.s, __shfl_sync(0xffffffffu, tok, src), __shfl_sync(0xffffffffu, h, src), lane);
      }
      tiles += j1 - j0;
      x += j1 - j0;
      j0 = 0;
      if (x < xend) rt_next(p, pre, HG, bq, u);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side

size_t ragged_tc_ws_floats(int D) { return (size_t)2 * RAGGED_TC_CTAS * (256 * D + 512); }

// [tokens][heads][D] rows `stride` elements apart, boxes of 64 x heads x rows
static bool make_tmap_rows_bf16(CUtensorMap* map, const void* ptr, int D, int heads, int tokens, long long stride,
                                int box_heads, int box_rows) {
  return make_tmap_bf16_3d(map, ptr, D, heads, tokens, 64, box_heads, box_rows, (uint64_t)stride);
}

template <int D, bool PAGED>
static cudaError_t ragged_tc(const CUtensorMap* m, const RaggedAttnParams& p, float* part, int* counters, int grid,
                             int hpc, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  const size_t smem = RtCfg<D>::SMEM + (size_t)(LLAMA_MAX_SEQS + 1) * 8;
  cudaError_t e = ensure_smem(attn_ragged_tc_kernel<D, PAGED>, smem, attr);
  if (e != cudaSuccess) return e;
  attn_ragged_tc_kernel<D, PAGED><<<grid, RT_THREADS, RtCfg<D>::SMEM + (size_t)(p.B + 1) * 8, st>>>(
      m[0], m[1], m[2], p, part, counters, hpc);
  return cudaGetLastError();
}

cudaError_t launch_attn_ragged_tc(const RaggedAttnParams& p, float* part, int* counters, int num_sms, cudaStream_t st) {
  const int hpc = prefill_heads_per_cta(p.H / p.Hkv);
  CUtensorMap m[3];
  bool ok = make_tmap_rows_bf16(&m[0], p.q, p.D, p.H, p.N, p.q_stride, hpc, 128 / hpc);
  if (p.tables) {
    const uint64_t rows = ((uint64_t)p.num_pages * p.Hkv) << p.page_shift;
    ok = ok && make_tmap_bf16(&m[1], p.k, rows, p.D, 1u << p.page_shift) &&
         make_tmap_bf16(&m[2], p.v, rows, p.D, 1u << p.page_shift);
  } else {
    ok = ok && make_tmap_rows_bf16(&m[1], p.k, p.D, p.Hkv, p.N, p.k_stride, 1, RT_KT) &&
         make_tmap_rows_bf16(&m[2], p.v, p.D, p.Hkv, p.N, p.v_stride, 1, RT_KT);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int grid = std::min(num_sms, RAGGED_TC_CTAS);
  if (p.D == 128)
    return p.tables ? ragged_tc<128, true>(m, p, part, counters, grid, hpc, st)
                    : ragged_tc<128, false>(m, p, part, counters, grid, hpc, st);
  return p.tables ? ragged_tc<64, true>(m, p, part, counters, grid, hpc, st)
                  : ragged_tc<64, false>(m, p, part, counters, grid, hpc, st);
}

}  // namespace llama
