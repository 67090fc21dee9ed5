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
// equal contiguous ranges (ragged.cuh), one per CTA and one CTA per SM, so the
// CTAs finish together whatever the lengths; a unit cut between CTAs leaves
// unnormalised partials (max, sum, O), merged in CTA order by the CTA that
// arrives last.
//   warp 0      TMA: Q (two boxes of 128 rows), then K(j), V(j) in turn through
//               a ring of 128-key stages (128-byte swizzle, no multicast); a
//               stage is 128 / page_size page boxes, a lane each. Pages past
//               the request's last one are read as out of range, i.e. zeros;
//   warps 1, 2  one thread each issues the MMAs of tile A / B: S = Q K(j)^T,
//               then O += P V in two parts (P of the first 96 and of the last
//               32 keys, read from TMEM, where the softmax wrote it over S),
//               then the next S. MMAs of one thread run in order, so S may
//               overwrite the P that the MMA before it reads, and the commit
//               behind S also tells the softmax that O is at rest;
//   warp 3      finds the CTA's segments in the list, a few ahead;
//   warps 4..7  softmax of tile A, one thread per row (its TMEM lane);
//   warps 8..11 softmax of tile B. While one tile's softmax runs, the tensor
//               core works on the other's.
//
// What bounds it: at long prompts the chain of one tile, S -> softmax -> P V ->
// next S. The MMAs of a 128 x 128 tile take 1029 cycles (64 each, measured) and
// its exponentials 1024 on the special-function unit (16 a cycle), but from the
// last MMA of a group to its commit pass another 420 cycles, so a tile's chain
// is about 1000 cycles of tensor core and 1700 of softmax, and A and B together
// reach 2500 to 3000 cycles per pair of tiles where the MMAs alone would take
// 2057. One prompt of 8192 tokens at 32/8 heads of 128: 468 us, 1175 TFLOP/s in a
// short burst; four of them 2.22 ms, 990 TFLOP/s, under the power limit (1.89 ms in
// single calls apart).
// Short prompts add what a unit costs besides its tiles (Q, the first S, the
// last P V, the way out of O: about 5 us, partly under its neighbours' work):
// 16 prompts of 17..2047 tokens at 32 heads 290 us in a short burst, 339 us call after
// call on new inputs. Measured on the way (bursts):
//  - one issuing thread picked by its lane number in place of elect.sync, and
//    one for both tiles: 635 us for the long prompt, 8 MMAs taking 423 cycles
//    to issue;
//  - 64-key steps with two S buffers a tile, so that S is never waited for: the
//    64-wide S MMAs read A as often and cost as much as 128-wide ones (529 us);
//  - two threads a row (16 softmax warps): 687 us;
//  - no turns at the exponentials: 655 us, both tiles falling into step;
//  - a quarter or half of the exponentials by a polynomial on the FMA pipe:
//    515 and 562 us against 509;
//  - rows stored by their own threads: 509 us against 484.
//
// A thread raises its running maximum only when a score passes it by more than
// 2^8 (O and the sum are then rescaled), and takes its weights 2^8 below it, so P <= 1.
//
// P is rounded to one bf16 for the product with V (fp32 sum of the unrounded
// values). Against the 64-bit form that leaves 2.0 to 2.3e-3 (relative, over all
// values) where rounding the output alone leaves 1.6 to 1.66e-3. With a second part of
// the remainder, as the contiguous prefill kernels have (attn_tc.cu), it is 1.6 to
// 1.66e-3, but the MMA work rises by half and the softmax has to make the parts: 8192
// tokens 468 -> 602 us (652 us there), ragged prompts 290 -> 421, chunks 171 -> 219, a mixed
// step 172 -> 213. The header states the rounding.
//
// V rows past the request's last key hold whatever the page or the next prompt
// holds; 0 x NaN is NaN in the MMA, so the softmax threads zero those rows of
// the last tile in shared memory before they hand over P. Infinities and NaN in V
// rows of keys in a unit's last tiles that not every row of it sees would reach the
// rows that do not see them the same way.
// Looking through V for them ahead of every P V cost 5 to 30 %, so it is done on
// demand: a segment with rows that are not finite, and with such values in V, is run
// again when the CTA's range is done. The softmax threads then put zeros for the values
// and note their keys, and a row that sees a noted key adds its values to O (with any
// weight above zero they are infinite or NaN all the same). So what such values cost is
// bounded by the call itself, however long the history: one prompt of 8192 tokens at
// 32/8 heads takes 470 us, 680 with an infinity at its start, 625 with one NaN in the
// middle, 1430 with nothing but NaN in V.
#include <algorithm>
#include <type_traits>

#include "ragged.cuh"

namespace llama {

namespace {
constexpr int RT_KT = 128;  // keys per tile (a K or V stage)
constexpr int RT_THREADS = 384;
constexpr int RT_SEGS = 3;  // segments queued ahead
constexpr int RT_MERGE = 6;      // what the merge of a cut unit costs, in tiles
constexpr int RT_FEW = 64;       // rows up to which all threads merge a cut unit, not a thread per row
constexpr int RT_LEADER = 128;  // first softmax thread
constexpr float RT_LOG2E = 1.4426950408889634f;
constexpr float RT_RESCALE = 8.0f;  // raise the running maximum only past 2^8
}  // namespace

// A segment: key tiles [j0, j1) of a unit (j1 = 0: the CTA's range ends here).
struct RtSeg {
  int b;                // request
  RaggedSeq s;
  int tok0, kvh, h0;    // first token and head of the unit's rows
  int j0, j1, whole;    // whole: all of the unit's key tiles
  int lim[2];           // key tiles that tiles A, B need (0 where the unit has no rows for B)
  int slot;             // where a partial of it goes
  int c0, c1, slot0;    // CTAs that share the unit, the slot of c0's partial
  int bit;              // of the segment in RtAgain
  unsigned odd[8];      // bit i: the i-th key behind those that every row sees has such values
};
// Segments to run again: a CTA's two cut units by their slots; whole ones share 512 bits (running
// one more of them again changes nothing).
struct RtAgain {
  int any, cut[2];
  unsigned whole[16];
};
static_assert(sizeof(RtAgain) <= 32 * 4, "zeroed by a warp");

template <int D>
struct RtCfg {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t HALF = RT_KT * 128;          // 128 rows x 64 bf16
  static constexpr uint32_t TILE = HALVES * HALF;        // a Q tile or a K or V stage
  static constexpr int STAGES = 131072 / TILE;           // 128 KB of ring
  static constexpr uint32_t S_COL = 0, O_COL = 256;      // S/P of A, B at 0, 128; O of A, B at 256, 384
  static constexpr int BARS = 2 * STAGES + 18 + 2 * RT_SEGS;
  static constexpr uint32_t OUT = 4096;                  // a softmax warp's 32 rows x 64 bf16 on their way out
  static constexpr size_t SMEM = 1024 + 2 * TILE + STAGES * TILE + 8 * OUT + BARS * 8 + 16 + RT_SEGS * sizeof(RtSeg) +
                                 sizeof(RtAgain) + 8 + (RT_PRE + 1) * 8;
  static_assert(SMEM + 256 <= 227 * 1024, "shared memory");
};

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
__device__ __forceinline__ void rt_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// this thread's stores have read their shared memory / have finished
__device__ __forceinline__ void rt_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void rt_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
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
// the N values that loads have been issued for are in (no use of them moves ahead of this)
template <int N>
__device__ __forceinline__ void rt_ld_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
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
__device__ __forceinline__ void rt_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void rt_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float rt_max3(float a, float b, float c) {  // NaN where one is
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float rt_max2(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float rt_ex2(float x) {  // 2^x on the special-function unit; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- V values that are not finite

// where the row of a key of the segment's request begins in V (-1: a page outside the pool, i.e. zeros)
template <bool PAGED>
__device__ __forceinline__ long long rt_v_row(const RaggedAttnParams& p, const RtSeg& w, int key, int D) {
  if (!PAGED) return (w.s.q0 + (long long)key) * p.v_stride + (long long)w.kvh * D;
  const int page = __ldg(p.tables + (size_t)w.b * p.max_pages + (key >> p.page_shift));
  if ((unsigned)page >= (unsigned)p.num_pages) return -1;
  return ((((long long)page * p.Hkv + w.kvh) << p.page_shift) + (key & ((1 << p.page_shift) - 1))) * D;
}
// of two bf16 values: bits 15 and 31 where the exponent is all ones
__device__ __forceinline__ uint32_t rt_odd2(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// Whether keys of the unit's tiles that not every row of it sees hold such values, by one warp
template <int D, bool PAGED>
__device__ __forceinline__ bool rt_v_odd(const RaggedAttnParams& p, const RtSeg& w, int lane) {
  const int all_see = w.s.kv - w.s.n_new + w.tok0 + 1;
  const int end = min(max(w.lim[0], w.lim[1]) * RT_KT, w.s.kv);
  uint32_t odd = 0;
#pragma unroll 2  // more loads at a time take registers that slow the producer (chunks over pages 5 %)
  for (int key = max(all_see, 0) + lane / (D / 8); key < end; key += 32 / (D / 8)) {
    const long long at = rt_v_row<PAGED>(p, w, key, D);
    const uint4 u = at < 0 ? make_uint4(0, 0, 0, 0)
                           : __ldg(reinterpret_cast<const uint4*>(static_cast<const bf16*>(p.v) + at) + lane % (D / 8));
    odd |= rt_odd2(u.x) | rt_odd2(u.y) | rt_odd2(u.z) | rt_odd2(u.w);
  }
  return __any_sync(0xffffffffu, odd != 0);
}
// Rows begin .. end - 1 of a V tile in the ring, by the threads of a tile: zeros for such values,
// notes of their keys (bits from row `begin` on; `notes` of them: later keys are seen by no row).
// The note comes before the zeros: the other tile's threads find either the value or its note.
template <int D>
__device__ __forceinline__ void rt_clean_v(uint8_t* v, int begin, int end, unsigned* odd, int notes, int r) {
#pragma unroll 1
  for (int k = max(begin, 0) * 8 + r; k < end * 8; k += 128)
#pragma unroll 1
    for (int hf = 0; hf < RtCfg<D>::HALVES; ++hf) {
      uint32_t* at = reinterpret_cast<uint32_t*>(v + hf * RtCfg<D>::HALF + k * 16);
      const int bit = (k >> 3) - begin;
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = at[e], found = rt_odd2(x);
        if (!found) continue;
        if (bit < notes) atomicOr(&odd[bit >> 5], 1u << (bit & 31));
        __threadfence_block();
        at[e] = x & ~((found >> 15) * 0xffffu);
      }
    }
}

// Values that were taken out of V come back to the rows of O that see their keys (a warp's 32 rows, in
// TMEM): a lane finds, for D / 32 columns, the first keys with +inf, -inf and NaN; a row that
// sees one of them adds it.
template <int D, bool PAGED>
__device__ __forceinline__ void rt_add_odd(const RaggedAttnParams& p, const RtSeg& w, uint32_t o_cols, int all_see, int last, int notes,
                                           int lane) {
  constexpr int N = D / 32, NONE = 0x7fffffff;
  int first[3][N];
#pragma unroll
  for (int k = 0; k < N; ++k) first[0][k] = first[1][k] = first[2][k] = NONE;
#pragma unroll 1
  for (int i0 = 0; i0 < notes; i0 += 4) {
    const unsigned bits = w.odd[i0 >> 5] >> (i0 & 31) & 15;
    if (bits == 0) continue;
    uint32_t x[4][N / 2];  // independent loads (8 keys at a time: ragged prompts 2 % slower, by registers)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long at = (bits >> i) & 1 ? rt_v_row<PAGED>(p, w, all_see + i0 + i, D) : -1;
#pragma unroll
      for (int k = 0; k < N / 2; ++k)
        x[i][k] = at < 0 ? 0u : __ldg(reinterpret_cast<const uint32_t*>(static_cast<const bf16*>(p.v) + at) + N / 2 * lane + k);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float2 pair = unpack_bf16x2(x[i][k / 2]);
        const float y = k % 2 ? pair.y : pair.x;
        const int key = all_see + i0 + i;
        if (y == INFINITY) first[0][k] = min(first[0][k], key);
        if (y == -INFINITY) first[1][k] = min(first[1][k], key);
        if (y != y) first[2][k] = min(first[2][k], key);
      }
  }
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float ov[32];
    rt_ld32(o_cols + c, ov);
    rt_ld_wait<32>(ov);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int from = (c + e) / N;
      if (__shfl_sync(0xffffffffu, first[0][e % N], from) <= last) ov[e] += INFINITY;
      if (__shfl_sync(0xffffffffu, first[1][e % N], from) <= last) ov[e] -= INFINITY;
      if (__shfl_sync(0xffffffffu, first[2][e % N], from) <= last) ov[e] += NAN;
    }
    __syncwarp();
    rt_st32(o_cols + c, reinterpret_cast<const uint32_t*>(ov));
  }
  rt_st_wait();
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(RT_THREADS, 1)
    attn_ragged_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                          const __grid_constant__ RaggedAttnParams p, float* __restrict__ part,
                          int* __restrict__ counters, int hpc) {
  using Cfg = RtCfg<D>;
  constexpr int ST = Cfg::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sKV = sQ + 2 * Cfg::TILE;
  uint8_t* sOut = sKV + ST * Cfg::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + 8 * Cfg::OUT);
  uint64_t* kv_full = bars;            // [ST] stage i % ST holds the i-th of K(0), V(0), K(1), V(1), ...
  uint64_t* kv_empty = kv_full + ST;   // [ST]
  uint64_t* q_full = kv_empty + ST;    // the segment's Q is in
  uint64_t* q_empty = q_full + 1;      // its last S has finished
  uint64_t* s_full = q_empty + 1;      // [g] S of tile A / B written (and every MMA of it before that finished)
  uint64_t* p_full = s_full + 2;       // [2 g + part] P of the first 96 / last 32 keys written over S
  uint64_t* o_full = p_full + 4;       // [g] the segment's last P V has finished
  uint64_t* o_free = o_full + 2;       // [g] O has been read
  volatile int* turns = reinterpret_cast<volatile int*>(o_free + 2);  // [4 g + quarter] key tiles whose exponentials are taken
  uint64_t* g_full = o_free + 6;        // [RT_SEGS] segment k is described in segs[k % RT_SEGS]
  uint64_t* g_empty = g_full + RT_SEGS;  // its readers (a warp each) have left it
  uint64_t* meet = g_empty + RT_SEGS;  // the softmax warps, at a cut unit
  uint64_t* walked = meet + 1;         // they are done with the range
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(walked + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_last = reinterpret_cast<int*>(tmem_slot + 2);
  RtSeg* segs = reinterpret_cast<RtSeg*>(tmem_slot + 4);
  RtAgain* again = reinterpret_cast<RtAgain*>(segs + RT_SEGS);
  // entries of one head group of the requests before i * per, per = ceil(B / RT_PRE)
  long long* pre = reinterpret_cast<long long*>((reinterpret_cast<uintptr_t>(again + 1) + 7) & ~uintptr_t(7));  // [RT_PRE + 1]
  __shared__ long long s_w[3 * RT_PRE / 32];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_rep = p.H / p.Hkv, groups = n_rep / hpc, HG = p.Hkv * groups;
  const int bq = 256 / hpc, bh = 128 / hpc;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 2);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], 128);
    for (int i = 0; i < 8; ++i) turns[i] = 0;
    mbar_init(meet, 256);
    mbar_init(walked, 8);
    for (int i = 0; i < RT_SEGS; ++i) {
      mbar_init(&g_full[i], 1);
      mbar_init(&g_empty[i], 11);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 128);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2 && lane < sizeof(RtAgain) / 4) reinterpret_cast<int*>(again)[lane] = 0;
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const bool units = rt_prefix<RT_KT, RT_MERGE>(p, bq, HG, pre, s_w);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // segment k, or false at the end of a pass (or after a timeout); given back by leave()
  auto enter = [&](int k) {
    return wait_or_abort(&g_full[k % RT_SEGS], (k / RT_SEGS) & 1, p.status, abort_flag) && segs[k % RT_SEGS].j1 > 0;
  };
  auto leave = [&](int k) { mbar_arrive(&g_empty[k % RT_SEGS]); };
  // After the segments of a pass, which end with one without tiles (it is left like the others, and
  // all counts run on): whether some are run again in a second one
  auto once_more = [&](int pass) {
    return pass == 0 && wait_or_abort(walked, 0, p.status, abort_flag) && *reinterpret_cast<volatile int*>(&again->any);
  };

  // 168 registers a thread at launch; the softmax threads hold a row of S and take
  // what the first four warps give back: 88 + 2 x 208 = 3 x 168
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ------------------------------------------------------------------ producer
      if (lane == 0) {
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
      }
      int i = 0, seg = 0, q = 0, pass = 0;  // ring slots, segments, Q tiles
      bool ok = true;
      do {
        while (ok && __all_sync(0xffffffffu, enter(seg))) {
          const RtSeg& w = segs[seg % RT_SEGS];
          const int kvh = w.kvh;
          if (lane == 0) {
            ok = wait_or_abort(q_empty, (q & 1) ^ 1, p.status, abort_flag);
            if (ok) {
              const int tiles = w.lim[1] ? 2 : 1;
              mbar_arrive_expect_tx(q_full, tiles * Cfg::TILE);
              for (int g = 0; g < tiles; ++g)
#pragma unroll
                for (int hf = 0; hf < Cfg::HALVES; ++hf)
                  rt_tma_3d(sQ + g * Cfg::TILE + hf * Cfg::HALF, &map_q, q_full, hf * 64, w.h0,
                            w.s.q0 + w.tok0 + g * bh);
            }
          }
          ok = __shfl_sync(0xffffffffu, (int)ok, 0);
          // lane -> (64-wide half, page of the tile); one box per lane
          const int ps = PAGED ? 1 << p.page_shift : RT_KT, boxes = Cfg::HALVES * (RT_KT / ps);
          const int hf = lane % Cfg::HALVES, pg = lane / Cfg::HALVES;
          const int n_pages = PAGED ? (w.s.kv + ps - 1) >> p.page_shift : 0;
          for (int j = w.j0; ok && j < w.j1; ++j) {
            int row = 0;
            if (PAGED && lane < boxes) {
              const int k = j * (RT_KT / ps) + pg;
              row = p.num_pages * p.Hkv * ps;  // out of range: zeros
              if (k < n_pages) {
                const int page = __ldg(p.tables + (size_t)w.b * p.max_pages + k);
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
                  rt_tma_3d(dst, map, &kv_full[st], hf * 64, kvh, w.s.q0 + j * RT_KT);
              }
            }
          }
          __syncwarp();
          if (lane == 0) leave(seg);
          ++seg;
          ++q;
        }
        if (lane == 0) leave(seg);
        ++seg;
      } while (ok && __all_sync(0xffffffffu, once_more(pass++)));
      // every copy lands before the CTA can retire
      if (lane == 0) {
        if (q > 0) mbar_wait(q_full, (q - 1) & 1, p.status);
        for (int k = (i > ST ? i - ST : 0); k < i; ++k) mbar_wait(&kv_full[k % ST], (k / ST) & 1, p.status);
      }
    } else if (warp <= 2) {
      if (elect_one()) {
        // ------------------------------------------------------------------ MMA issuer of tile A / B
        constexpr uint32_t idesc_s = make_idesc_bf16(128, RT_KT);
        constexpr uint32_t idesc_pv = make_idesc_bf16(128, D) | (1u << 16);  // B (= V) N-major
        const int g = warp - 1;
        const uint32_t qa = smem_u32(sQ + g * Cfg::TILE), kv = smem_u32(sKV);
        const uint32_t sd = tmem + Cfg::S_COL + g * 128, od = tmem + Cfg::O_COL + g * 128;
        int i = 0, seg = 0, q = 0, pass = 0;  // ring slots, segments, Q tiles
        int pc = 0, oc = 0;                   // P tiles, segments with work
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t par) { return ok = ok && wait_or_abort(bar, par & 1, p.status, abort_flag); };
        auto issue_s = [&](int st) {
          const uint32_t ka = kv + st * Cfg::TILE;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * Cfg::HALF + (kk & 3) * 32;
            tc_mma_bf16(sd, make_sw128_desc(qa + off), make_sw128_desc(ka + off), idesc_s, kk > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[g]);
        };
        do {
          for (; ok && enter(seg); ++seg) {
            const int j0 = segs[seg % RT_SEGS].j0, j1 = segs[seg % RT_SEGS].j1;
            const int jl = min(j1, segs[seg % RT_SEGS].lim[g]);  // this tile has work on [j0, jl)
            leave(seg);
            if (!wait(q_full, q++) || !wait(&kv_full[i % ST], i / ST)) break;
            tc_fence_after();
            if (j0 < jl) {
              issue_s(i % ST);
              tc_commit(&kv_empty[i % ST]);
            } else {
              mbar_arrive(&kv_empty[i % ST]);
            }
            if (jl - j0 <= 1) tc_commit(q_empty);
            for (int j = j0; j < j1; ++j, i += 2) {
              const int vs = (i + 1) % ST, ks = (i + 2) % ST;  // ring stages of V(j), K(j + 1)
              if (!wait(&kv_full[vs], (i + 1) / ST)) break;
              if (j < jl) {
                if (j == j0 && !wait(&o_free[g], oc++ ^ 1)) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  if (!wait(&p_full[2 * g + h], pc)) break;
                  tc_fence_after();
#pragma unroll
                  for (int kk = 6 * h; kk < 6 + 2 * h; ++kk)
                    rt_mma_ts(od, sd + kk * 8, rt_desc_n(kv + vs * Cfg::TILE + kk * 2048, Cfg::HALF), idesc_pv,
                              (j > j0 || kk > 0) ? 1u : 0u);
                }
                if (!ok) break;
                ++pc;
                if (j + 1 == jl) tc_commit(&o_full[g]);
              }
              if (j + 1 < j1) {
                if (!wait(&kv_full[ks], (i + 2) / ST)) break;
                if (j + 1 < jl) {
                  issue_s(ks);
                  tc_commit(&kv_empty[ks]);
                } else {
                  mbar_arrive(&kv_empty[ks]);
                }
              }
              if (j < jl)
                tc_commit(&kv_empty[vs]);
              else
                mbar_arrive(&kv_empty[vs]);
              if (j + 2 == jl) tc_commit(q_empty);  // the segment's last S has been issued
            }
          }
          leave(seg++);
        } while (ok && once_more(pass++));
        // every MMA finishes before TMEM is freed: the softmax warps wait for all of
        // them (o_full), except after a timeout
        if (!ok) {
          tc_commit(q_empty);
          const uint64_t t0 = global_timer_ns();
          while (global_timer_ns() - t0 < LLAMA_WAIT_LIMIT_NS / 16) {
          }
        }
      }
    } else {
      // ------------------------------------------------------------------ scheduler
      const long long W = pre[RT_PRE] * HG, G = min((long long)gridDim.x, W), cta = blockIdx.x;
      RtWalk w;
      w.units = units;
      w.x = cta < G ? rt_begin(cta, W, G) : 0;
      w.end = cta < G ? rt_begin(cta + 1, W, G) : 0;
      const long long xbeg = w.x;
      rt_start<RT_KT>(p, pre, HG, bq, w);
      for (int k = 0, pass = 0, at = 0;;) {  // segments handed out, passes, segments of the range
        const bool more = rt_segment<RT_KT>(bq, w);
        const bool whole = w.j0 == 0 && w.j1 == w.n;
        const int bit = at++ & 511, cut = w.xs <= xbeg ? 0 : 1;
        if (more && pass == 1 && !(whole ? (again->whole[bit >> 5] >> (bit & 31)) & 1 : again->cut[cut])) {
          rt_advance(p, HG, bq, w);
          continue;
        }
        if (!__all_sync(0xffffffffu, wait_or_abort(&g_empty[k % RT_SEGS], ((k / RT_SEGS) & 1) ^ 1, p.status, abort_flag))) break;
        RtSeg& q = segs[k % RT_SEGS];
        if (lane == 0) {
          q.j1 = 0;
          if (more) {
            q.b = w.b;
            q.s = w.s;
            q.tok0 = w.t * bq;
            q.kvh = w.zl / groups;
            q.h0 = q.kvh * n_rep + (w.zl - q.kvh * groups) * hpc;
            q.j0 = w.j0;
            q.j1 = w.j1;
            q.whole = whole;
            q.lim[0] = w.lim[0];
            q.lim[1] = w.lim[1];
            // a CTA has at most two cut units, one at either end of its range
            q.slot = (int)(2 * cta + cut);
            const long long x0 = w.xs + RT_UNIT;  // the unit's first tile
            q.c0 = (int)rt_own(x0, W, G);
            q.c1 = (int)rt_own(x0 + w.n - 1, W, G);
            q.slot0 = 2 * q.c0 + (w.xs <= rt_begin(q.c0, W, G) ? 0 : 1);
            q.bit = bit;
#pragma unroll
            for (int e = 0; e < 8; ++e) q.odd[e] = 0;
          }
        }
        __syncwarp();
        // rows of a whole unit that see such values alone are right as they are
        if (pass == 0 || !more || !whole || rt_v_odd<D, PAGED>(p, q, lane)) {
          if (lane == 0) mbar_arrive(&g_full[k % RT_SEGS]);
          ++k;
        }
        if (more) {
          rt_advance(p, HG, bq, w);
          continue;
        }
        if (!__all_sync(0xffffffffu, once_more(pass++))) break;
        at = 0;
        w.x = xbeg;
        rt_start<RT_KT>(p, pre, HG, bq, w);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // -------------------------------------------------------------------- softmax
    int sc = 0, oc = 0;                // S tiles taken, segments with work
    int n = 0;                         // key tiles walked (ring slots 2 n, 2 n + 1)
    bool ok = true;
    int seg = 0, met = 0;
    // One pass over the range. The second one is code of its own, from values that the compiler
    // does not see to be the first one's: sharing them cost the first pass 3 to 12 %.
    auto walk = [&](auto second, int tid, uint32_t tmem, int hpc) {
      constexpr bool CLEAN = decltype(second)::value;
      if (CLEAN) asm volatile("" : "+r"(tid), "+r"(tmem), "+r"(hpc));
      const int warp = tid >> 5, lane = tid & 31, bh = 128 / hpc;
      const int g = warp >= 8 ? 1 : 0;
      const int quarter = warp & 3, r = quarter * 32 + lane;  // row of the tile = TMEM lane
      const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
      const uint32_t s_cols = lanes + Cfg::S_COL + g * 128, o_cols = lanes + Cfg::O_COL + g * 128;
      const float sl2 = rsqrtf((float)D) * RT_LOG2E;
      const uint64_t scale2 = rt_f2(sl2, sl2);
      const int pos_l = r / hpc, hl = r - pos_l * hpc;
      const int stride = 256 * D + 512;  // floats of one partial
      uint8_t* out = sOut + (warp - 4) * Cfg::OUT;
      // (maximum, 1 / sum) of row rr of a merged unit of few rows, where the row's warp has its way out
      auto few = [&](int rr) { return reinterpret_cast<float2*>(sOut + (rr >> 5) * Cfg::OUT) + (rr & 31); };
      static_assert(RT_FEW <= 128, "rows of tile A");
      const int tok_end = 31 / hpc + quarter * 32 / hpc;  // the warp's last token, in the tile
      // The warps of A and B on one scheduler take maximum and exponentials in turn: A's tile
      // n after B's n - 1, B's n after A's n. Left alone they fall into step, both at the
      // exponentials and then both waiting for the tensor core. No more than a hint: a
      // warp that has waited long goes on.
      auto my_turn = [&] {
        const int want = g == 0 ? n : n + 1;
        for (int i = 0; i < 256 && turns[4 * (g ^ 1) + quarter] < want; ++i) {
        }
        __syncwarp();
      };
      auto meet_all = [&] {
        mbar_arrive(meet);
        ok = wait_or_abort(meet, met++ & 1, p.status, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
      };
      auto pass_turn = [&](int tiles) {
        n += tiles;
        turns[4 * g + quarter] = n;
      };
      for (; ok && __all_sync(0xffffffffu, enter(seg)); ++seg) {
        RtSeg& w = segs[seg % RT_SEGS];
        const int lim = w.lim[g], j1 = w.j1, jl = min(j1, lim);  // this tile's rows have work on [j0, jl)
        const int tok = w.tok0 + g * bh + pos_l, kv_len = w.s.kv;
        const int all_see = w.s.kv - w.s.n_new + w.tok0 + 1;  // keys that every row of the unit sees
        // last key this row sees (rows past the last token follow it)
        const int last = min(w.s.kv - w.s.n_new + min(tok, w.s.n_new - 1), w.s.kv - 1);
        const bool live = __any_sync(0xffffffffu, tok < w.s.n_new);  // else no row of this warp is anyone's
        float m_used = -INFINITY, l = 0.f;
        for (int j = w.j0; ok && j < jl; ++j) {
          ok = wait_or_abort(&s_full[g], sc & 1, p.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++sc;
          tc_fence_after();
          const int key0 = j * RT_KT;
          const bool clean = CLEAN && key0 + RT_KT > all_see;
          if (key0 + RT_KT > kv_len || clean) {
            // V rows past the last key: zeros, before the MMA may read them
            const int vs = 2 * n + 1, row0 = min(max(kv_len - key0, 0), RT_KT);
            ok = wait_or_abort(&kv_full[vs % ST], (vs / ST) & 1, p.status, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint8_t* v = sKV + (vs % ST) * Cfg::TILE + row0 * 128;
            const int n16 = (RT_KT - row0) * 8;  // 16-byte pieces of one half
            for (int k = r; k < n16 * Cfg::HALVES; k += 128)
              *reinterpret_cast<uint4*>(v + (k / n16) * Cfg::HALF + (k % n16) * 16) = make_uint4(0, 0, 0, 0);
            if (clean) rt_clean_v<D>(sKV + (vs % ST) * Cfg::TILE, all_see - key0, row0, w.odd, 2 * bh - 1, r);
            fence_proxy_async_smem();
          }
          if (live) {
            // p = 2^(s log2(e) / sqrt(D) - m) -> bf16 pairs over this row's S
            float s[RT_KT];
#pragma unroll
            for (int c = 0; c < RT_KT; c += 32) rt_ld32(s_cols + c, s + c);
            rt_ld_wait<RT_KT>(s);
            const int seen = last - key0;  // keys 0 .. seen of the tile
            if (__any_sync(0xffffffffu, RT_KT - 1 > seen)) {
#pragma unroll
              for (int c = 0; c < RT_KT; ++c) s[c] = c > seen ? -INFINITY : s[c];
            }
            my_turn();
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < RT_KT - 4; c += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) mx[k] = rt_max3(mx[k], s[c + 2 * k], s[c + 2 * k + 1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = rt_max2(mx[k], s[RT_KT - 4 + k]);
            const float mt = rt_max3(rt_max2(mx[0], mx[1]), mx[2], mx[3]) * sl2;  // log2 units
            if (j == w.j0) {
              m_used = mt;
            } else if (__any_sync(0xffffffffu, !(mt <= m_used + RT_RESCALE))) {
              // S(j) was issued behind P(j - 1) V(j - 1), so O is at rest
              const float m_new = rt_max2(m_used, mt);
              const float alpha = m_new == -INFINITY ? 1.f : rt_ex2(m_used - m_new);
              l *= alpha;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float ov[32];
                rt_ld32(o_cols + c, ov);
                rt_ld_wait<32>(ov);
#pragma unroll
                for (int k = 0; k < 32; ++k) ov[k] *= alpha;
                rt_st32(o_cols + c, reinterpret_cast<const uint32_t*>(ov));
              }
              m_used = m_new;
            }
            const float m_ref = m_used == -INFINITY ? 0.f : -RT_RESCALE - m_used;
            const uint64_t negm2 = rt_f2(m_ref, m_ref);
            uint64_t ls[2] = {rt_f2(0.f, 0.f), rt_f2(0.f, 0.f)};
            auto weights = [&](int c0) {
              uint32_t pp[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float p0, p1;
                rt_split(rt_fma2(rt_f2(s[c0 + 2 * k], s[c0 + 2 * k + 1]), scale2, negm2), p0, p1);
                p0 = rt_ex2(p0);
                p1 = rt_ex2(p1);
                ls[k & 1] = rt_add2(ls[k & 1], rt_f2(p0, p1));
                pp[k] = pack_bf16x2(p0, p1);
              }
              rt_st16(s_cols + c0 / 2, pp);
            };
            weights(0);
            weights(32);
            weights(64);
            rt_st_wait();
            tc_fence_before();
            mbar_arrive(&p_full[2 * g]);
            weights(96);
            pass_turn(1);
            float a0, a1, b0, b1;
            rt_split(ls[0], a0, a1);
            rt_split(ls[1], b0, b1);
            l += (a0 + a1) + (b0 + b1);
            rt_st_wait();
            tc_fence_before();
          } else {
            pass_turn(1);
            mbar_arrive(&p_full[2 * g]);
          }
          mbar_arrive(&p_full[2 * g + 1]);
        }
        pass_turn(j1 - max(jl, w.j0));
        const bool work = w.j0 < jl;
        if (ok && work) {
          ok = wait_or_abort(&o_full[g], oc & 1, p.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          ++oc;
          tc_fence_after();
        }
        if (!ok) break;
        if (CLEAN && work) rt_add_odd<D, PAGED>(p, w, o_cols, all_see, last, 2 * bh - 1, lane);
        const int h = w.h0 + hl;
        const bool store = tok < w.s.n_new && lim > 0;
        bf16* dst = reinterpret_cast<bf16*>(p.o) + ((size_t)(w.s.q0 + tok) * p.H + h) * D;
        bool bad = false;  // the row's result is not finite
        const int rows = (int)min((long long)(w.s.n_new - w.tok0) * hpc, 256LL);  // rows of the request in the unit
        if (w.whole) {
          const float inv = last < 0 ? 0.f : 1.f / l;  // a row without keys is zero
          // 32 rows of the request leave as boxes of 64 columns, by way of shared memory:
          // a thread's stores to its own row touch a sector each
          const bool boxes = w.tok0 + g * bh + tok_end < w.s.n_new;
          if (work && boxes) {
#pragma unroll 1
            for (int c = 0; c < D; c += 64) {
              float ov[64];
              rt_ld32(o_cols + c, ov);
              rt_ld32(o_cols + c + 32, ov + 32);
              rt_ld_wait<64>(ov);
              if (c + 64 >= D) {
                tc_fence_before();
                mbar_arrive(&o_free[g]);
              }
              uint4 u[8];
#pragma unroll
              for (int e = 0; e < 64; ++e) {
                ov[e] = last < 0 ? 0.f : ov[e] * inv;
                bad |= !(fabsf(ov[e]) < INFINITY);
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) store8(reinterpret_cast<bf16*>(&u[e]), ov + 8 * e);
              if (lane == 0) rt_store_wait_read();  // the box before has been read
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4*>(out + lane * 128 + ((e ^ (lane & 7)) << 4)) = u[e];
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0)
                rt_store_3d(&map_o, out, c, w.h0, w.s.q0 + w.tok0 + g * bh + tok_end - 31 / hpc);
            }
          } else if (work) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float ov[32];
              rt_ld32(o_cols + c, ov);
              rt_ld_wait<32>(ov);
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
          if (__any_sync(0xffffffffu, bad && store && l > 0.f) && !CLEAN && lane == 0) {
            atomicOr(&again->whole[w.bit >> 5], 1u << (w.bit & 31));
            again->any = 1;
          }
        } else {
          // partial: O as [D / 4][256 rows] float4, then (max, sum) per row
          float* pp = part + (size_t)w.slot * stride;
          const int row = g * 128 + r;
          if (work) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float ov[32];
              rt_ld32(o_cols + c, ov);
              rt_ld_wait<32>(ov);
#pragma unroll
              for (int e = 0; e < 32; ++e) bad |= !(fabsf(ov[e]) < INFINITY);
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
          if (__any_sync(0xffffffffu, bad && store && l > 0.f) && !CLEAN && lane == 0)
            again->cut[w.slot & 1] = again->any = 1;
          meet_all();
          if (!ok) break;
          if (!CLEAN && again->cut[w.slot & 1]) {  // handed over when it has been run again
            __syncwarp();
            if (lane == 0) leave(seg);
            continue;
          }
          const int c0 = w.c0, c1 = w.c1;
          if (tid == RT_LEADER) *s_last = atomic_add_acq_rel(&counters[c0], 1) == c1 - c0;
          meet_all();
          if (!ok) break;
          if (*s_last) {
            if (rows <= RT_FEW) {  // few() lies there
              if (lane == 0) rt_store_wait_read();
              __syncwarp();
            }
            // partials of CTAs c0 .. c1 in that order; c0 holds the unit in its second slot
            // unless its range starts inside it, the others in their first
            const int slot0 = w.slot0;
            // batches of independent loads: one by one they would cost an L2 round trip each
            auto slot = [&](int c) { return part + (size_t)(c == c0 ? slot0 : 2 * c) * stride; };
            if (store) {
              float mm = -INFINITY, ll = 0.f;
              for (int c = c0; c <= c1; c += 16) {
                float2 v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  v[k] = c + k <= c1 ? __ldcg(reinterpret_cast<const float2*>(slot(c + k) + 256 * D) + row)
                                     : make_float2(-INFINITY, 0.f);
                float mn = mm;
#pragma unroll
                for (int k = 0; k < 16; ++k) mn = fmaxf(mn, v[k].x);
                if (mm != -INFINITY) ll *= rt_ex2(mm - mn);
                mm = mn;
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  if (v[k].x != -INFINITY) ll += v[k].y * rt_ex2(v[k].x - mm);
              }
              const float inv = last < 0 ? 0.f : 1.f / ll;
              if (rows <= RT_FEW) *few(row) = make_float2(mm, last < 0 ? -1.f : inv);  // -1: a row without keys
#pragma unroll 1
              for (int d = 0; rows > RT_FEW && d < D; d += 32) {
                float acc[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) acc[e] = 0.f;
#pragma unroll 1
                for (int c = c0; c <= c1; c += 2) {
                  float m_c[2];
                  float4 v[2][8];
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    const float* pc = slot(min(c + k, c1));
                    m_c[k] = c + k <= c1 ? __ldcg(reinterpret_cast<const float2*>(pc + 256 * D) + row).x : -INFINITY;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[k][e] = __ldcg(reinterpret_cast<const float4*>(pc) + (d / 4 + e) * 256 + row);
                  }
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    if (m_c[k] == -INFINITY) continue;  // no weight there (and perhaps no O)
                    const float f = rt_ex2(m_c[k] - mm);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                      acc[4 * e] += v[k][e].x * f;
                      acc[4 * e + 1] += v[k][e].y * f;
                      acc[4 * e + 2] += v[k][e].z * f;
                      acc[4 * e + 3] += v[k][e].w * f;
                    }
                  }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) acc[e] = last < 0 ? 0.f : acc[e] * inv;
#pragma unroll
                for (int e = 0; e < 32; e += 8) store8(dst + d + e, acc + e);
              }
            }
            if (rows <= RT_FEW) {
              // few rows (single tokens, short chunks over long histories): 4 columns of a row at
              // a time, over all threads; with a thread per row the merge of 18 partials of 16
              // rows took most of 42 us
              meet_all();
              if (!ok) break;
              for (int it = tid - RT_LEADER; it < rows * (D / 4); it += 256) {
                const int c4 = it / rows, rr = it - c4 * rows;
                const float2 mi = *few(rr);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c = c0; c <= c1; c += 8) {
                  float m_c[8];
                  float4 v[8];
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    const float* pc = slot(min(c + k, c1));
                    m_c[k] = c + k <= c1 ? __ldcg(reinterpret_cast<const float2*>(pc + 256 * D) + rr).x : -INFINITY;
                    v[k] = __ldcg(reinterpret_cast<const float4*>(pc) + c4 * 256 + rr);
                  }
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    if (m_c[k] == -INFINITY) continue;  // no weight there (and perhaps no O)
                    const float f = rt_ex2(m_c[k] - mi.x);
                    acc.x += v[k].x * f;
                    acc.y += v[k].y * f;
                    acc.z += v[k].z * f;
                    acc.w += v[k].w * f;
                  }
                }
                float y[4] = {acc.x * mi.y, acc.y * mi.y, acc.z * mi.y, acc.w * mi.y};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (mi.y == -1.f) y[e] = 0.f;
                store4(reinterpret_cast<bf16*>(p.o) +
                           ((size_t)(w.s.q0 + w.tok0 + rr / hpc) * p.H + w.h0 + rr % hpc) * D + 4 * c4,
                       y);
              }
            }
            if (tid == RT_LEADER) counters[c0] = 0;  // re-armed for the next launch
          }
          meet_all();  // s_last is written again by the next cut segment
          if (!ok) break;
        }
        __syncwarp();
        if (lane == 0) leave(seg);
      }
    };
    walk(std::false_type{}, tid, tmem, hpc);
    if (lane == 0) {
      leave(seg);
      mbar_arrive(walked);
    }
    ++seg;
    if (lane == 0) rt_store_wait();
    if (ok && __all_sync(0xffffffffu, once_more(0))) {
      walk(std::true_type{}, tid, tmem, hpc);
      if (lane == 0) rt_store_wait();
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
  const size_t smem = RtCfg<D>::SMEM;
  cudaError_t e = ensure_smem(attn_ragged_tc_kernel<D, PAGED>, smem, attr);
  if (e != cudaSuccess) return e;
  attn_ragged_tc_kernel<D, PAGED><<<grid, RT_THREADS, smem, st>>>(
      m[0], m[1], m[2], m[3], p, part, counters, hpc);
  return cudaGetLastError();
}

cudaError_t launch_attn_ragged_tc(const RaggedAttnParams& p, float* part, int* counters, int num_sms, cudaStream_t st) {
  const int hpc = prefill_heads_per_cta(p.H / p.Hkv);
  CUtensorMap m[4];
  bool ok = make_tmap_rows_bf16(&m[0], p.q, p.D, p.H, p.N, p.q_stride, hpc, 128 / hpc) &&
            make_tmap_rows_bf16(&m[3], p.o, p.D, p.H, p.N, (long long)p.H * p.D, hpc, 32 / hpc);
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
