// Attention of single new tokens over a paged cache (bf16): for request b with kv
// keys and query head h, softmax_j(q.k_j / sqrt(D)) V over all of them.
//
// What bounds it: every K and V row is read once for the heads that share it, so
// HBM. A unit is (request, kv head, group of hpc query heads), its history
// ceil(kv / 64) key tiles. The tiles of all units, unit-major, form one list that
// is cut into equal contiguous ranges, one per CTA and two CTAs per SM, so each CTA
// streams the same number of bytes whatever the lengths, and 192 KB per SM are in
// flight. A unit cut between CTAs leaves partials (max, sum, O), merged in CTA
// order by the CTA that arrives last.
//   warp 4      TMA: the K and V tiles of the range through a 3-stage ring
//               (128-byte swizzle, no multicast), a page box per lane; pages past
//               the request's last one are read as out of range, i.e. zeros;
//   warps 0..3  warp w takes keys 16 w .. 16 w + 15 of every tile on the warp-level
//               bf16 MMA (HBM-bound: it keeps up) with its own running maximum, sum
//               and O; P is split into two bf16 parts (~16 bits kept, rd_split). At the
//               end of a segment the four states merge in the ring stage of its last tile.
// V rows past the last key hold whatever the page holds, and 0 x NaN is NaN in the
// MMA: the warp that owns them zeroes them in shared memory first.
//
// Measured: 32 requests of 1024..8128 tokens at 32/8 heads (497 MB) 89 us, 5.6 TB/s, 85 %
// of a copy; one request of some 600 tokens at 32 heads 9.4 us, bound by the chain
// lengths, table, tiles, partials, merge.
//
// A CTA keeps 12 bytes of shared memory per request. At head_dim 128 that leaves room for two
// CTAs per SM up to about 1300 requests; beyond them one is resident, and half the bytes are
// in flight: 1.2 M keys of 2 kv heads in 1290 requests 219 us (5.6 TB/s), in 1320 322 us
// (3.8), in 3900 391 us (3.1). At head_dim 64 two always fit (246, 242 and 276 us).
#include "ragged.cuh"

#include <algorithm>

namespace llama {

namespace {
constexpr int RD_KT = 64;      // keys per tile
constexpr int RD_STAGES = 3;
constexpr float RD_LOG2E = 1.4426950408889634f;
}  // namespace

// element (row, col) of a 64-row x 64-column bf16 box written with 128-byte swizzling
__device__ __forceinline__ uint32_t rd_sw(uint32_t box, int row, int col) {
  return box + row * 128 + ((((col >> 3) ^ (row & 7)) & 7) << 4) + (col & 7) * 2;
}
__device__ __forceinline__ float rd_quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float rd_quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// tiles of one unit of a request with kv keys (one for a token that sees none: its
// row is written as zeros), 0 for a request without a new token (kv = -1)
__host__ __device__ __forceinline__ int rd_tiles(int kv) { return kv < 0 ? 0 : kv == 0 ? 1 : (kv - 1) / RD_KT + 1; }

struct RdUnit {
  int b, zl;  // request, unit inside the request (kv head * groups + group)
  int t;      // tile inside the unit
};
// pb[b]: tiles of one head group of the requests before b
__host__ __device__ __forceinline__ RdUnit rd_locate(const long long* pb, const int* kvs, int B, int HG, long long x) {
  int lo = 0, hi = B - 1;  // the last b whose tiles begin at or before x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pb[mid] * HG <= x) lo = mid; else hi = mid - 1;
  }
  RdUnit u;
  u.b = lo;
  const long long off = x - pb[lo] * HG;
  const int n = rd_tiles(kvs[lo]);
  u.zl = (int)(off / n);
  u.t = (int)(off - (long long)u.zl * n);
  return u;
}

// rows [r0, r1) of a V tile become zeros, by one warp
template <int HALVES>
__device__ __forceinline__ void rd_zero_rows(uint8_t* v, int r0, int r1, int lane) {
  const int n16 = (r1 - r0) * 8;
  for (int e = lane; e < n16 * HALVES; e += 32)
    *reinterpret_cast<uint4*>(v + (e / n16) * 8192 + r0 * 128 + (e % n16) * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();  // before the next TMA write into the stage
  __syncwarp();
}

// floats of one partial: O [hpc][D], then (max, sum) per head, padded to 16 bytes
__host__ __device__ __forceinline__ int rd_part_stride(int hpc, int D) { return hpc * D + ((2 * hpc + 3) & ~3); }

// Transpose of an 8 x 8 matrix of 16-bit values held as a warp fragment (thread
// t holds row t / 4, columns 2 (t % 4), 2 (t % 4) + 1): afterwards thread t holds
// row t / 4 of the transpose.
__device__ __forceinline__ uint32_t rd_transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// (a, b) >= 0 as hi + lo, pairs of bf16: the upper halves, and the remainders rounded to
// bf16 (the sum is off by at most 2^-16 of the value). Both parts of a weight above zero are above zero, so an
// infinite V stays infinite in both products: a part rounded to nearest may be zero or
// negative, and 0 x inf and inf - inf are NaN. 2^-126 stands in for a remainder of zero, below
// what a sum of such values shows; a weight of zero stays zero.
__device__ __forceinline__ void rd_split(float a, float b, uint32_t& hi, uint32_t& lo) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  hi = __byte_perm(ua, ub, 0x7632);
  lo = pack_bf16x2(a - __uint_as_float(ua & 0xffff0000u), b - __uint_as_float(ub & 0xffff0000u));
  uint32_t least;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(least) : "r"(hi), "r"(0x00800080u));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(least));
}

// NARROW (a unit serves at most 8 query heads): the scores are computed as
// S^T = K q^T with the 16 keys of a warp as the MMA rows and the heads as its
// 8 columns, and the output as O^T = V^T P^T (head dimension as rows), so no
// MMA row is spent on a missing head: half the MMAs and exponentials of the
// heads-as-rows form, which the wider groups (9..16 heads) keep.
template <int D, bool NARROW>
__global__ void __launch_bounds__(160, 2)
    attn_ragged_decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                              const RaggedAttnParams p, float* __restrict__ part, int* __restrict__ counters, int hpc) {
  constexpr uint32_t TB = RD_KT * D * 2;  // one K or one V tile
  constexpr int HALVES = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(base + RD_STAGES * 2 * TB);
  uint64_t* empty = full + RD_STAGES;
  long long* pb = reinterpret_cast<long long*>(empty + RD_STAGES);  // [B + 1]
  int* kvs = reinterpret_cast<int*>(pb + p.B + 1);               // [B] keys, or -1
  __shared__ float s_m[64], s_l[64];  // (max, sum) of [4 warps][16 rows] at a segment's merge
  __shared__ int s_last;
  __shared__ long long s_w[5];
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.B, n_rep = p.H / p.Hkv, groups = n_rep / hpc, HG = p.Hkv * groups;
  const int pstride = rd_part_stride(hpc, D);

  if (tid == 0) {
    for (int i = 0; i < RD_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    s_abort = 0;
    fence_barrier_init();
  }
  {
    const int per = (B + 159) / 160, b0 = min(tid * per, B), b1 = min(b0 + per, B);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      RaggedSeq s;
      ragged_seq(p, b, s, blockIdx.x == 0);
      kvs[b] = s.n_new ? s.kv : -1;
      sum += rd_tiles(kvs[b]);
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
      pb[b] = x;
      x += rd_tiles(kvs[b]);
      if (b == B - 1) pb[B] = x;
    }
    __syncthreads();
  }
  const long long W = pb[B] * HG, G = min((long long)gridDim.x, W), cta = blockIdx.x;
  const long long sbeg = cta < G ? rt_begin(cta, W, G) : 0, send = cta < G ? rt_begin(cta + 1, W, G) : 0;

  if (warp == 4) {
    // ---------------------------------------------------------------- producer
    if (sbeg >= send) return;
    if (lane == 0) {
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_v);
    }
    RdUnit u = rd_locate(pb, kvs, B, HG, sbeg);
    // lane -> (K or V, 64-wide half, page box of the tile)
    const int ps = min(1 << p.page_shift, RD_KT), per = RD_KT / ps;
    const int kv = lane & 1, hf = (lane >> 1) % HALVES, pg = (lane >> 1) / HALVES;
    const bool mine = lane < 2 * HALVES * per;
    int j = 0;
    bool ok = true;
    for (long long x = sbeg; x < send; ++x, ++j) {
      const int n_keys = kvs[u.b], kvh = u.zl / groups, key = u.t * RD_KT + pg * ps;
      int row = (p.num_pages * p.Hkv) << p.page_shift;  // out of range: zeros
      if (mine && key < n_keys) {
        const int page = __ldg(p.tables + (size_t)u.b * p.max_pages + (key >> p.page_shift));
        if ((unsigned)page < (unsigned)p.num_pages)
          row = ((page * p.Hkv + kvh) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
        else
          atomicOr(p.status, LLAMA_DEV_PAGE_RANGE);
      }
      const int st = j % RD_STAGES;
      ok = wait_or_abort(&empty[st], ((j / RD_STAGES) & 1) ^ 1, p.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[st], 2 * TB);
      __syncwarp();
      if (mine) tma_load_2d(base + st * 2 * TB + kv * TB + hf * 8192 + pg * ps * 128, kv ? &map_v : &map_k, &full[st], hf * 64, row);
      if (++u.t == rd_tiles(n_keys)) {
        u.t = 0;
        if (++u.zl == HG) {
          u.zl = 0;
          do ++u.b;
          while (u.b < B - 1 && kvs[u.b] < 0);
        }
      }
    }
    // no copy may be in flight when the CTA exits
    if (lane == 0)
      for (int i = (j > RD_STAGES ? j - RD_STAGES : 0); i < j; ++i)
        mbar_wait(&full[i % RD_STAGES], (i / RD_STAGES) & 1, p.status);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int g = lane >> 2, qd = lane & 3;
  const float sl2 = rsqrtf((float)D) * RD_LOG2E;
  const bool rv0 = g < hpc, rv1 = g + 8 < hpc;  // rows g, g + 8 are heads of the group
  int j = 0;
  long long x = sbeg;
  bf16* const o = reinterpret_cast<bf16*>(p.o);
  while (x < send) {
    const RdUnit u = rd_locate(pb, kvs, B, HG, x);
    const int L = kvs[u.b], n_u = rd_tiles(L);
    const int seg_len = (int)min(send - x, (long long)(n_u - u.t));
    const int kvh = u.zl / groups, grp = u.zl - kvh * groups;
    const int h0 = kvh * n_rep + grp * hpc;
    const size_t tok = p.cu[u.b];
    const bf16* q = reinterpret_cast<const bf16*>(p.q) + tok * p.q_stride + (size_t)h0 * D;
    bf16* dst = o + (tok * p.H + h0) * D;

    int st = 0;  // the ring stage of the segment's last tile
    if constexpr (NARROW) {
      // ---- keys as MMA rows: thread (g, qd) holds heads 2qd, 2qd + 1 of keys g and g + 8
      uint32_t qb[D / 16][2];  // B fragments of q^T: head g, d pairs 2qd (+8) of each 16-d step
      {
        const bf16* r0 = q + (rv0 ? g : 0) * D;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qb[kk][0] = rv0 ? *reinterpret_cast<const uint32_t*>(r0 + 16 * kk + 2 * qd) : 0u;
          qb[kk][1] = rv0 ? *reinterpret_cast<const uint32_t*>(r0 + 16 * kk + 8 + 2 * qd) : 0u;
        }
      }
      float ot[D / 16][4];  // O^T: rows d = 16 i + g (+8), columns heads 2qd, 2qd + 1
#pragma unroll
      for (int i = 0; i < D / 16; ++i) ot[i][0] = ot[i][1] = ot[i][2] = ot[i][3] = 0.f;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2qd, 2qd + 1
      for (int i = 0; i < seg_len; ++i, ++j) {
        st = j % RD_STAGES;
        const bool ok = wait_or_abort(&full[st], (j / RD_STAGES) & 1, p.status, abort_flag);
        const int key0 = (u.t + i) * RD_KT + 16 * warp;  // first of this warp's 16 keys
        if (__all_sync(0xffffffffu, ok) && key0 < L) {
          const uint32_t kb = smem_u32(base + st * 2 * TB), vb = kb + TB;
          if (key0 + 16 > L) rd_zero_rows<HALVES>(base + st * 2 * TB + TB, 16 * warp + L - key0, 16 * warp + 16, lane);
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int key = 16 * warp + (lane & 7) + 8 * ((lane >> 3) & 1);
            const int d = 16 * kk + 8 * (lane >> 4);
            uint32_t a[4];
            ldmatrix_x4(a, rd_sw(kb + (d >> 6) * 8192, key, d & 63));
            mma_bf16_16816(s, a, qb[kk]);
          }
          // scale; keys at or past the history's end are masked
          s[0] = key0 + g >= L ? -INFINITY : s[0] * sl2;
          s[1] = key0 + g >= L ? -INFINITY : s[1] * sl2;
          s[2] = key0 + g + 8 >= L ? -INFINITY : s[2] * sl2;
          s[3] = key0 + g + 8 >= L ? -INFINITY : s[3] * sl2;
          float mx0 = fmaxf(s[0], s[2]), mx1 = fmaxf(s[1], s[3]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {  // over the 8 key rows g
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
          }
          const float old0 = m0, old1 = m1;
          m0 = fmaxf(m0, mx0);
          m1 = fmaxf(m1, mx1);
          // 0 stands in for a maximum of -inf (scores of -inf alone)
          const float mn0 = m0 == -INFINITY ? 0.f : m0, mn1 = m1 == -INFINITY ? 0.f : m1;
          const float sc0 = exp2f(old0 - mn0), sc1 = exp2f(old1 - mn1);
          l0 *= sc0;
          l1 *= sc1;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            ot[c][0] *= sc0;
            ot[c][1] *= sc1;
            ot[c][2] *= sc0;
            ot[c][3] *= sc1;
          }
          s[0] = exp2f(s[0] - mn0);
          s[1] = exp2f(s[1] - mn1);
          s[2] = exp2f(s[2] - mn0);
          s[3] = exp2f(s[3] - mn1);
          l0 += s[0] + s[2];
          l1 += s[1] + s[3];
          // P^T as B fragments (key pairs 2qd (+8), head g), hi + lo bf16 parts:
          // transpose the [key][head] fragments of keys 0-7 and 8-15
          uint32_t h01, l01, h23, l23;
          rd_split(s[0], s[1], h01, l01);
          rd_split(s[2], s[3], h23, l23);
          const uint32_t bh[2] = {rd_transpose(h01), rd_transpose(h23)};
          const uint32_t bl[2] = {rd_transpose(l01), rd_transpose(l23)};
          // O^T += V^T P^T over this warp's 16 keys; V^T fragments by transposed loads of V
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const int mi = lane >> 3;
            const int key = 16 * warp + 8 * (mi >> 1) + (lane & 7);
            const int d = 16 * c + 8 * (mi & 1);
            uint32_t a[4];
            ldmatrix_x4_trans(a, rd_sw(vb + (d >> 6) * 8192, key, d & 63));
            mma_bf16_16816(ot[c], a, bh);
            mma_bf16_16816(ot[c], a, bl);
          }
        }
        if (i + 1 < seg_len) {  // the segment's last stage is released after the merge below
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
        }
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
      }
      // this warp's state -> [warp][head][D] in the stage of the segment's last tile
      asm volatile("bar.sync 1, 128;" ::: "memory");
      float* so = reinterpret_cast<float*>(base + st * 2 * TB);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        so[(warp * 16 + 2 * qd) * D + 16 * c + g] = ot[c][0];
        so[(warp * 16 + 2 * qd + 1) * D + 16 * c + g] = ot[c][1];
        so[(warp * 16 + 2 * qd) * D + 16 * c + g + 8] = ot[c][2];
        so[(warp * 16 + 2 * qd + 1) * D + 16 * c + g + 8] = ot[c][3];
      }
      if (g == 0) {
        s_m[warp * 16 + 2 * qd] = m0;
        s_m[warp * 16 + 2 * qd + 1] = m1;
        s_l[warp * 16 + 2 * qd] = l0;
        s_l[warp * 16 + 2 * qd + 1] = l1;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
    } else {
      uint32_t qa[D / 16][4];
      {
        const bf16* r0 = q + (rv0 ? g : 0) * D;
        const bf16* r1 = q + (rv1 ? g + 8 : 0) * D;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qa[kk][0] = rv0 ? *reinterpret_cast<const uint32_t*>(r0 + 16 * kk + 2 * qd) : 0u;
          qa[kk][1] = rv1 ? *reinterpret_cast<const uint32_t*>(r1 + 16 * kk + 2 * qd) : 0u;
          qa[kk][2] = rv0 ? *reinterpret_cast<const uint32_t*>(r0 + 16 * kk + 8 + 2 * qd) : 0u;
          qa[kk][3] = rv1 ? *reinterpret_cast<const uint32_t*>(r1 + 16 * kk + 8 + 2 * qd) : 0u;
        }
      }
      float oacc[D / 8][4];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) oacc[c][0] = oacc[c][1] = oacc[c][2] = oacc[c][3] = 0.f;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

      for (int i = 0; i < seg_len; ++i, ++j) {
        st = j % RD_STAGES;
        const bool ok = wait_or_abort(&full[st], (j / RD_STAGES) & 1, p.status, abort_flag);
        const int key0 = (u.t + i) * RD_KT + 16 * warp;  // first of this warp's 16 keys
        if (__all_sync(0xffffffffu, ok) && key0 < L) {
          const uint32_t kb = smem_u32(base + st * 2 * TB), vb = kb + TB;
          if (key0 + 16 > L) rd_zero_rows<HALVES>(base + st * 2 * TB + TB, 16 * warp + L - key0, 16 * warp + 16, lane);
          float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int mi = lane >> 3;
            const int key = 16 * warp + 8 * (mi >> 1) + (lane & 7);
            const int d = 16 * kk + 8 * (mi & 1);
            uint32_t bf[4];
            ldmatrix_x4(bf, rd_sw(kb + (d >> 6) * 8192, key, d & 63));
            const uint32_t b0[2] = {bf[0], bf[1]}, b1[2] = {bf[2], bf[3]};
            mma_bf16_16816(s[0], qa[kk], b0);
            mma_bf16_16816(s[1], qa[kk], b1);
          }
          float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
          for (int jn = 0; jn < 2; ++jn)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v = s[jn][e] * sl2;
              if (key0 + 8 * jn + 2 * qd + (e & 1) >= L) v = -INFINITY;
              s[jn][e] = v;
              if (e < 2)
                mx0 = fmaxf(mx0, v);
              else
                mx1 = fmaxf(mx1, v);
            }
          const float old0 = m0, old1 = m1;
          m0 = fmaxf(m0, rd_quad_max(mx0));
          m1 = fmaxf(m1, rd_quad_max(mx1));
          // 0 stands in for a maximum of -inf (scores of -inf alone)
          const float mn0 = m0 == -INFINITY ? 0.f : m0, mn1 = m1 == -INFINITY ? 0.f : m1;
          const float sc0 = exp2f(old0 - mn0), sc1 = exp2f(old1 - mn1);
          l0 *= sc0;
          l1 *= sc1;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            oacc[c][0] *= sc0;
            oacc[c][1] *= sc0;
            oacc[c][2] *= sc1;
            oacc[c][3] *= sc1;
          }
#pragma unroll
          for (int jn = 0; jn < 2; ++jn) {
            s[jn][0] = exp2f(s[jn][0] - mn0);
            s[jn][1] = exp2f(s[jn][1] - mn0);
            s[jn][2] = exp2f(s[jn][2] - mn1);
            s[jn][3] = exp2f(s[jn][3] - mn1);
            l0 += s[jn][0] + s[jn][1];
            l1 += s[jn][2] + s[jn][3];
          }
          // O += P V over this warp's 16 keys, P as hi + lo bf16 parts
          uint32_t ph[4], pl[4];
          rd_split(s[0][0], s[0][1], ph[0], pl[0]);
          rd_split(s[0][2], s[0][3], ph[1], pl[1]);
          rd_split(s[1][0], s[1][1], ph[2], pl[2]);
          rd_split(s[1][2], s[1][3], ph[3], pl[3]);
#pragma unroll
          for (int jd = 0; jd < D / 8; jd += 2) {
            const int mi = lane >> 3;
            const int key = 16 * warp + 8 * (mi & 1) + (lane & 7);
            const int d = 8 * (jd + (mi >> 1));
            uint32_t bf[4];
            ldmatrix_x4_trans(bf, rd_sw(vb + (d >> 6) * 8192, key, d & 63));
            const uint32_t b0[2] = {bf[0], bf[1]}, b1[2] = {bf[2], bf[3]};
            mma_bf16_16816(oacc[jd], ph, b0);
            mma_bf16_16816(oacc[jd], pl, b0);
            mma_bf16_16816(oacc[jd + 1], ph, b1);
            mma_bf16_16816(oacc[jd + 1], pl, b1);
          }
        }
        if (i + 1 < seg_len) {  // the segment's last stage is released after the merge below
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
        }
      }
      l0 = rd_quad_sum(l0);
      l1 = rd_quad_sum(l1);
      // this warp's state -> [warp][head][D] in the stage of the segment's last tile
      asm volatile("bar.sync 1, 128;" ::: "memory");
      float* so = reinterpret_cast<float*>(base + st * 2 * TB);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        *reinterpret_cast<float2*>(so + (warp * 16 + g) * D + 8 * c + 2 * qd) = make_float2(oacc[c][0], oacc[c][1]);
        *reinterpret_cast<float2*>(so + (warp * 16 + g + 8) * D + 8 * c + 2 * qd) =
            make_float2(oacc[c][2], oacc[c][3]);
      }
      if (qd == 0) {
        s_m[warp * 16 + g] = m0;
        s_m[warp * 16 + g + 8] = m1;
        s_l[warp * 16 + g] = l0;
        s_l[warp * 16 + g + 8] = l1;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    // Merge the four warps' states, held in the stage of the segment's last
    // tile, which every warp has finished reading: [4 warps][16 rows][D] floats
    // fill its 2 x 64 x D bf16 exactly; the (max, sum) pairs are in s_m, s_l.
    float* sm_o = reinterpret_cast<float*>(base + st * 2 * TB);
    const long long P = pb[u.b] * HG + (long long)u.zl * n_u;  // the unit's first tile
    const bool whole = u.t == 0 && seg_len == n_u;
    // Partial state of this CTA for a split unit: slot 2 cta when the unit began
    // before this range (the range's first segment), else slot 2 cta + 1 (the
    // unit runs past the range's end: its last segment).
    float* pp = part + (size_t)(2 * cta + (P <= sbeg ? 0 : 1)) * pstride;
    for (int e = tid; e < hpc * D; e += 128) {
      const int r = e / D, d = e - r * D;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_m[w * 16 + r]);
      float acc = 0.f, ll = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float mw = s_m[w * 16 + r];
        const float f = mw == -INFINITY ? 0.f : exp2f(mw - mm);  // a warp without valid keys in the segment
        acc += sm_o[(w * 16 + r) * D + d] * f;
        ll += s_l[w * 16 + r] * f;
      }
      if (whole) {  // the whole unit is in this range: normalise and store
        dst[r * D + d] = __float2bfloat16_rn(L > 0 ? acc / ll : 0.f);
      } else {
        __stcg(pp + r * D + d, acc);
        if (d == 0) __stcg(reinterpret_cast<float2*>(pp + hpc * D + 2 * r), make_float2(mm, ll));
      }
    }
    fence_proxy_async_smem();  // these generic writes come before the next TMA write into the stage
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (lane == 0) mbar_arrive(&empty[st]);

    if (!whole) {
      const int c0 = (int)rt_own(P, W, G), c1 = (int)rt_own(P + n_u - 1, W, G);
      // a CTA begins at most one unit that runs past its range: its counter serves it
      if (tid == 0) s_last = (atomic_add_acq_rel(&counters[c0], 1) == c1 - c0);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (s_last) {
        // The last contributor merges the partials of CTAs c0 .. c1 in that
        // order: m = max m_c, l = sum l_c 2^(m_c - m), o = sum o_c 2^(m_c - m) / l.
        // CTA c0 holds the unit in its second slot unless its range starts at
        // the unit; every later contributor holds it in its first slot.
        const int slot0 = 2 * c0 + (rt_begin(c0, W, G) == P ? 0 : 1);
        for (int e = tid; e < hpc * D / 4; e += 128) {
          const int r = (4 * e) / D, d = 4 * e - r * D;
          // batches of independent loads: one by one they would cost an L2 round trip each
          auto slot = [&](int c) { return part + (size_t)(c == c0 ? slot0 : 2 * c) * pstride; };
          float mm = -INFINITY;
          for (int c = c0; c <= c1; c += 16) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = c + k <= c1 ? __ldcg(slot(c + k) + hpc * D + 2 * r) : -INFINITY;
#pragma unroll
            for (int k = 0; k < 16; ++k) mm = fmaxf(mm, v[k]);
          }
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          float ll = 0.f;
          for (int c = c0; c <= c1; c += 8) {
            float2 ml[8];
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float* pc = slot(min(c + k, c1));
              ml[k] = __ldcg(reinterpret_cast<const float2*>(pc + hpc * D + 2 * r));
              v[k] = __ldcg(reinterpret_cast<const float4*>(pc + r * D + d));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (c + k > c1) continue;
              const float f = ml[k].x == -INFINITY ? 0.f : exp2f(ml[k].x - mm);
              ll += ml[k].y * f;
              acc.x += v[k].x * f;
              acc.y += v[k].y * f;
              acc.z += v[k].z * f;
              acc.w += v[k].w * f;
            }
          }
          const float il = 1.f / ll;
          uint2 w;
          w.x = pack_bf16x2(acc.x * il, acc.y * il);
          w.y = pack_bf16x2(acc.z * il, acc.w * il);
          *reinterpret_cast<uint2*>(dst + r * D + d) = w;
        }
        if (tid == 0) counters[c0] = 0;  // re-armed for the next launch
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");  // s_last is rewritten by the next segment
    }
    x += seg_len;
  }
}

// ------------------------------------------------------------------ host side

static size_t rd_smem(int D, int B) {
  return 1024 + (size_t)RD_STAGES * 2 * RD_KT * D * 2 + 2 * RD_STAGES * 8 + (size_t)(B + 1) * 8 + (size_t)B * 4;
}

// Host walk of the split, as check_ragged_list
static bool check_decode_list(const RaggedAttnParams& p, int grid) {
  const int hpc = decode_heads_per_cta(p.H / p.Hkv), HG = p.H / hpc;
  if (p.H % hpc) return false;
  std::vector<long long> pb(p.B + 1, 0);
  std::vector<int> kvs(p.B);
  long long units = 0;
  for (int b = 0; b < p.B; ++b) {
    RaggedSeq s;
    ragged_seq(p, b, s, false);
    kvs[b] = s.n_new ? s.kv : -1;
    pb[b + 1] = pb[b] + rd_tiles(kvs[b]);
    units += s.n_new ? HG : 0;
  }
  const long long W = pb[p.B] * HG, G = W < grid ? W : grid;
  std::vector<char> slot_used(2 * (size_t)grid, 0), counter_used(grid, 0);
  long long done = 0, next = 0;
  for (int cta = 0; cta < G; ++cta) {
    const long long sbeg = rt_begin(cta, W, G), send = rt_begin(cta + 1, W, G);
    if (sbeg != next) return false;
    next = send;
    for (long long x = sbeg; x < send;) {
      const RdUnit u = rd_locate(pb.data(), kvs.data(), p.B, HG, x);
      const int n = rd_tiles(kvs[u.b]);
      if (n < 1 || u.zl < 0 || u.zl >= HG || u.t < 0 || u.t >= n || pb[u.b] * HG + (long long)u.zl * n + u.t != x) return false;
      const long long len = n - u.t < send - x ? n - u.t : send - x, P = x - u.t;
      if (u.t > 0 || len < n) {
        const int c0 = (int)rt_own(P, W, G), c1 = (int)rt_own(P + n - 1, W, G), slot = 2 * cta + (P <= sbeg ? 0 : 1);
        if (cta < c0 || cta > c1 || (u.t == 0) != (cta == c0) || (u.t + len == n) != (cta == c1)) return false;
        if (slot != (cta == c0 ? 2 * c0 + (rt_begin(c0, W, G) == P ? 0 : 1) : 2 * cta) || slot_used[slot]) return false;
        slot_used[slot] = 1;
        if (cta == c0 && counter_used[c0]) return false;
        counter_used[c0] = 1;
      }
      done += u.t + len == n;
      x += len;
    }
  }
  return next == W && done == units;
}

// The lists of all three attention kernels for these lengths (host memory), on so many SMs
bool check_ragged_plans(const int* cu, const int* kv_lens, int B, int N, int max_kv, int H, int Hkv, int num_sms) {
  RaggedAttnParams p = {};
  int page = 0;
  p.cu = cu;
  p.kv_lens = kv_lens;
  p.tables = &page;  // lengths as of a paged call
  p.B = B;
  p.N = N;
  p.max_new = N;
  p.H = H;
  p.Hkv = Hkv;
  p.page_shift = 4;
  p.max_pages = (max_kv + 15) / 16;
  bool ok = true;
  for (bool units : {false, true}) {
    ok = ok && check_ragged_list<128>(p, 256, std::min(num_sms, RAGGED_TC_CTAS), units);
    for (int per_sm : {3, 2}) ok = ok && check_ragged_list<64>(p, 32, std::min(num_sms, RAGGED_F32_CTAS / 3) * per_sm, units);
  }
  p.max_new = 1;  // requests with more are skipped there
  return ok && check_decode_list(p, std::min(2 * num_sms, RAGGED_DECODE_CTAS));
}

size_t ragged_decode_ws_floats(int D) { return (size_t)2 * RAGGED_DECODE_CTAS * rd_part_stride(16, D); }

template <int D, bool NARROW>
static cudaError_t ragged_decode(const CUtensorMap* m, const RaggedAttnParams& p, float* part, int* counters, int grid,
                                 int hpc, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  cudaError_t e = ensure_smem(attn_ragged_decode_kernel<D, NARROW>, rd_smem(D, LLAMA_MAX_SEQS), attr);
  if (e != cudaSuccess) return e;
  attn_ragged_decode_kernel<D, NARROW><<<grid, 160, rd_smem(D, p.B), st>>>(m[0], m[1], p, part, counters, hpc);
  return cudaGetLastError();
}

cudaError_t launch_attn_ragged_decode(const RaggedAttnParams& p, float* part, int* counters, int num_sms,
                                      cudaStream_t st) {
  const int hpc = decode_heads_per_cta(p.H / p.Hkv);
  const uint64_t rows = ((uint64_t)p.num_pages * p.Hkv) << p.page_shift;
  const uint32_t box = std::min(1u << p.page_shift, (uint32_t)RD_KT);
  CUtensorMap m[2];
  if (!make_tmap_bf16(&m[0], p.k, rows, p.D, box) || !make_tmap_bf16(&m[1], p.v, rows, p.D, box))
    return cudaErrorInvalidValue;
  const int grid = std::min(2 * num_sms, RAGGED_DECODE_CTAS);
  if (hpc <= 8)
    return p.D == 128 ? ragged_decode<128, true>(m, p, part, counters, grid, hpc, st)
                      : ragged_decode<64, true>(m, p, part, counters, grid, hpc, st);
  return p.D == 128 ? ragged_decode<128, false>(m, p, part, counters, grid, hpc, st)
                    : ragged_decode<64, false>(m, p, part, counters, grid, hpc, st);
}

}  // namespace llama
