// Causal attention of packed rows over a paged cache or over packed keys, in fp32 on
// the CUDA cores: softmax_j(q.k_j / sqrt(D)) V over the keys j <= p of each row.
//
// What bounds it: the FMA pipe where rows share their keys (2 D products per row and
// key), HBM for single tokens. A unit is 32 query rows of one (request, kv head): hpc
// query heads (the largest power of two up to 8 dividing n_rep) x 32 / hpc positions;
// it walks 64-key tiles up to its last position. The tiles of all units form one list,
// cut evenly over the CTAs (ragged.cuh), because fp32 models are small: a few short
// prompts have fewer units than the GPU has SMs. A unit cut between CTAs leaves
// partials (max, sum, O), merged in CTA order by the CTA that arrives last.
//
// 128 threads, thread (ty, tx) of 8 x 16: scores of rows 4 ty .. + 3 with keys tx + 16 k,
// then outputs of the same rows with columns 4 tx .. + 3 (+ 64): each 16-byte read of
// shared memory serves 8 products. K(j + 1) is copied while P(j) V(j) runs and V(j + 1)
// while the scores of j + 1 are taken (cp.async; keys past the last one are zeros).
//
// Measured at 4/2 heads of 64: 7 prompts of 5..509 tokens 23.6 us (four CTAs per SM, which
// spill: 32 us), 5 requests of up to 761 keys with up to 61 new tokens 17.5 us; of a CTA's
// time there 3 us pass before it knows its range and 3 until its first tile is in, the rest
// is one or two tiles and the merge of the cut unit.
//
// 0 x NaN and 0 x inf are NaN: where a tile has keys that not every row of the unit sees
// (at most its last two), the threads look through the V rows of those keys that they
// copied, put zeros for values that are not finite and note the keys; rows that see such
// a key add its values at the end (with any weight above zero they are infinite or NaN
// all the same).
#include "ragged.cuh"

#include <algorithm>

namespace llama {

namespace {
constexpr int RF_KT = 64;       // keys per tile
constexpr int RF_ROWS = 32;     // query rows per unit
constexpr int RF_THREADS = 128;
constexpr int RF_MERGE = 3;     // what the merge of a cut unit costs, in tiles
constexpr float RF_LOG2E = 1.4426950408889634f;
}  // namespace

template <int D>
struct RfCfg {
  static constexpr int LD = D + 4;      // row stride of Q and K: 16 rows on distinct banks
  static constexpr int LDP = RF_KT + 4;
  static constexpr int FLOATS = RF_ROWS * LD + RF_KT * LD + RF_KT * D + RF_ROWS * LDP;
  static constexpr size_t SMEM = FLOATS * 4;
  static constexpr int PER_SM = D == 64 ? 3 : 2;  // resident CTAs (a fourth fits in shared memory, but spills registers)
};

__device__ __forceinline__ void rf_copy16(void* dst, const void* src, int bytes) {  // bytes 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void rf_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void rf_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(RF_THREADS, RfCfg<D>::PER_SM)
    attn_ragged_f32_kernel(const RaggedAttnParams p, float* __restrict__ part, int* __restrict__ counters, int hpc) {
  using Cfg = RfCfg<D>;
  constexpr int LD = Cfg::LD, LDP = Cfg::LDP, NC = D / 64;
  extern __shared__ float4 rf_smem[];
  float* sQ = reinterpret_cast<float*>(rf_smem);
  float* sK = sQ + RF_ROWS * LD;
  float* sV = sK + RF_KT * LD;
  float* sP = sV + RF_KT * D;
  __shared__ long long pre[RT_PRE + 1];
  __shared__ long long s_w[3 * RT_PRE / 32];
  __shared__ int s_last;
  __shared__ unsigned s_odd;  // bit i: the i-th key behind those that every row sees has V values that are not finite

  const int tid = threadIdx.x, warp = tid >> 5, tx = tid & 15, ty = tid >> 4;
  const int n_rep = p.H / p.Hkv, groups = n_rep / hpc, HG = p.Hkv * groups, bq = RF_ROWS / hpc;
  const int stride = RF_ROWS * D + 2 * RF_ROWS;  // floats of one partial
  const float sl2 = rsqrtf((float)D) * RF_LOG2E;
  RtWalk w;
  w.units = rt_prefix<RF_KT, RF_MERGE>(p, bq, HG, pre, s_w);
  const long long W = pre[RT_PRE] * HG, G = min((long long)gridDim.x, W), cta = blockIdx.x;
  w.x = cta < G ? rt_begin(cta, W, G) : 0;
  w.end = cta < G ? rt_begin(cta + 1, W, G) : 0;
  const long long xbeg = w.x;
  rt_start<RF_KT>(p, pre, HG, bq, w);
  for (; rt_segment<RF_KT>(bq, w); rt_advance(p, HG, bq, w)) {
    const int kvh = w.zl / groups, h0 = kvh * n_rep + (w.zl - kvh * groups) * hpc, tok0 = w.t * bq;
    // a thread copies 16 bytes of the same column of every LR-th row
    constexpr int LR = RF_THREADS * 4 / D;
    const int lrow = tid / (D / 4), lcol = (tid % (D / 4)) * 4;
    const int all_see = w.s.kv - w.s.n_new + tok0 + 1;  // keys that every row of the unit sees
    auto load = [&](float* dst, int ld, const void* src, long long row_stride, int j) {
      const float* from = static_cast<const float*>(src) + lcol;
      const int* table = p.tables + (size_t)w.b * p.max_pages;
#pragma unroll 8
      for (int i = 0; i < RF_KT / LR; ++i) {
        const int r = lrow + i * LR, key = j * RF_KT + r;
        bool have = key < w.s.kv;
        const float* at = from;
        if (p.tables) {
          const int page = have ? __ldg(table + (key >> p.page_shift)) : 0;
          if ((unsigned)page >= (unsigned)p.num_pages) {
            have = false;
            atomicOr(p.status, LLAMA_DEV_PAGE_RANGE);
          }
          // rows of all pages number fewer than 2^31
          const int row = ((page * p.Hkv + kvh) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
          if (have) at += (size_t)row * D;
        } else if (have) {
          at += (size_t)(w.s.q0 + key) * row_stride + kvh * D;
        }
        rf_copy16(dst + r * ld + lcol, at, have ? 16 : 0);
      }
      rf_commit();
    };
    __syncthreads();  // shared memory of the segment before has been read
    if (tid == 0) s_odd = 0;
#pragma unroll
    for (int i = 0; i < RF_ROWS / LR; ++i) {
      const int r = lrow + i * LR, tok = tok0 + r / hpc;
      const bool have = tok < w.s.n_new;
      const float* at = static_cast<const float*>(p.q) + lcol;
      if (have) at += (size_t)(w.s.q0 + tok) * p.q_stride + (h0 + r % hpc) * D;
      rf_copy16(sQ + r * LD + lcol, at, have ? 16 : 0);
    }
    load(sK, LD, p.k, p.k_stride, w.j0);
    load(sV, D, p.v, p.v_stride, w.j0);

    const bool live = tok0 + 8 * warp / hpc < w.s.n_new;  // a row of this warp is someone's
    int last[4];                                          // last key each row sees
    float m[4], l[4];
    uint64_t o2[4][2 * NC];  // outputs, in pairs of columns
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = tok0 + (4 * ty + i) / hpc;
      last[i] = min(w.s.kv - w.s.n_new + min(tok, w.s.n_new - 1), w.s.kv - 1);
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) o2[i][c] = 0;
    }
    for (int j = w.j0; j < w.j1; ++j) {
      rf_wait_but_one();
      __syncthreads();  // Q, K(j) in; P(j - 1), V(j - 1) read
      float s[4][4];
      if (live) {
        uint64_t s2[4][4];  // sums over even and over odd d
#pragma unroll
        for (int i = 0; i < 4; ++i) s2[i][0] = s2[i][1] = s2[i][2] = s2[i][3] = 0;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          ulonglong2 q[4], k[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const ulonglong2*>(sQ + (4 * ty + i) * LD + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) k[i] = *reinterpret_cast<const ulonglong2*>(sK + (tx + 16 * i) * LD + d);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) s2[i][c] = rt_fma2(q[i].x, k[c].x, rt_fma2(q[i].y, k[c].y, s2[i][c]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float even, odd;
            rt_split(s2[i][c], even, odd);
            s[i][c] = even + odd;
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float mt = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            s[i][c] = j * RF_KT + tx + 16 * c > last[i] ? -INFINITY : s[i][c] * sl2;
            mt = fmaxf(mt, s[i][c]);
          }
#pragma unroll
          for (int x = 8; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
          const float mn = fmaxf(m[i], mt), ref = mn == -INFINITY ? 0.f : mn, a = exp2f(m[i] - ref);
          m[i] = mn;
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float e = exp2f(s[i][c] - ref);
            sum += e;
            sP[(4 * ty + i) * LDP + tx + 16 * c] = e;
          }
          l[i] = l[i] * a + sum;  // of this thread's keys
#pragma unroll
          for (int c = 0; c < 2 * NC; ++c) o2[i][c] = rt_mul2(o2[i][c], rt_f2(a, a));
        }
      }
      __syncthreads();  // K(j) read
      if (j + 1 < w.j1)
        load(sK, LD, p.k, p.k_stride, j + 1);
      else
        rf_commit();
      rf_wait_but_one();
      if ((j + 1) * RF_KT > all_see) {
#pragma unroll 4
        for (int i = 0; i < RF_KT / LR; ++i) {
          const int r = lrow + i * LR, bit = j * RF_KT + r - all_see;
          float4* at = reinterpret_cast<float4*>(sV + r * D + lcol);
          const float4 v = *at;
          const float any = fmaf(v.x, 0.f, v.y * 0.f) + fmaf(v.z, 0.f, v.w * 0.f);  // NaN where one is not finite
          if (bit >= 0 && !(any == 0.f)) {
            if (bit < 32) atomicOr(&s_odd, 1u << bit);  // later keys are seen by no row
            *at = make_float4(fabsf(v.x) < INFINITY ? v.x : 0.f, fabsf(v.y) < INFINITY ? v.y : 0.f,
                              fabsf(v.z) < INFINITY ? v.z : 0.f, fabsf(v.w) < INFINITY ? v.w : 0.f);
          }
        }
      }
      __syncthreads();  // V(j), P(j) in
      if (live) {
#pragma unroll 4
        for (int k = 0; k < RF_KT; k += 4) {
          float4 pr[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4*>(sP + (4 * ty + i) * LDP + k);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sV + (k + kk) * D + 64 * c + 4 * tx);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float e = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
                o2[i][2 * c] = rt_fma2(rt_f2(e, e), v.x, o2[i][2 * c]);
                o2[i][2 * c + 1] = rt_fma2(rt_f2(e, e), v.y, o2[i][2 * c + 1]);
              }
            }
        }
      }
      __syncthreads();  // V(j) read
      if (j + 1 < w.j1)
        load(sV, D, p.v, p.v_stride, j + 1);
      else
        rf_commit();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);

    float o[4][4 * NC];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) rt_split(o2[i][c], o[i][2 * c], o[i][2 * c + 1]);
    if (s_odd) {
#pragma unroll 1
      for (unsigned bits = s_odd; bits; bits &= bits - 1) {
        const int key = all_see + __ffs(bits) - 1;
        const float* at = static_cast<const float*>(p.v) + 4 * tx;
        if (p.tables) {
          const int page = __ldg(p.tables + (size_t)w.b * p.max_pages + (key >> p.page_shift));
          if ((unsigned)page >= (unsigned)p.num_pages) continue;
          at += (size_t)(((page * p.Hkv + kvh) << p.page_shift) + (key & ((1 << p.page_shift) - 1))) * D;
        } else {
          at += (size_t)(w.s.q0 + key) * p.v_stride + kvh * D;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(at + 64 * c));
          const float odd[4] = {fabsf(v.x) < INFINITY ? 0.f : v.x, fabsf(v.y) < INFINITY ? 0.f : v.y,
                                fabsf(v.z) < INFINITY ? 0.f : v.z, fabsf(v.w) < INFINITY ? 0.f : v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][4 * c + e] += key <= last[i] ? odd[e] : 0.f;
        }
      }
    }
    // normalise and store row i of this thread (columns 4 tx + 64 c)
    auto finish = [&](int i, float sum) {
      const int r = 4 * ty + i, tok = tok0 + r / hpc;
      if (tok >= w.s.n_new) return;
      float* dst = static_cast<float*>(p.o) + ((size_t)(w.s.q0 + tok) * p.H + h0 + r % hpc) * D;
      const float inv = 1.f / sum;
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c) o[i][c] = last[i] < 0 ? 0.f : o[i][c] * inv;  // a row without keys is zero
#pragma unroll
      for (int c = 0; c < NC; ++c) store4(dst + 64 * c + 4 * tx, o[i] + 4 * c);
    };
    if (w.j0 == 0 && w.j1 == w.n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) finish(i, l[i]);
    } else {
      // a CTA has at most two cut units, one at either end of its range
      float* pp = part + (size_t)(2 * cta + (w.xs <= xbeg ? 0 : 1)) * stride;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (tok0 + r / hpc >= w.s.n_new) continue;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          __stcg(reinterpret_cast<float4*>(pp + r * D + 64 * c + 4 * tx),
                 make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]));
        if (tx == 0) __stcg(reinterpret_cast<float2*>(pp + RF_ROWS * D) + r, make_float2(m[i], l[i]));
      }
      __syncthreads();
      const long long x0 = w.xs + RT_UNIT;  // the unit's first tile
      const int c0 = (int)rt_own(x0, W, G), c1 = (int)rt_own(x0 + w.n - 1, W, G);
      if (tid == 0) s_last = atomic_add_acq_rel(&counters[c0], 1) == c1 - c0;
      __syncthreads();
      if (s_last) {
        const int slot0 = 2 * c0 + (w.xs <= rt_begin(c0, W, G) ? 0 : 1);
// batches of independent loads: one by one they would cost an L2 round trip each
        auto slot = [&](int c) { return part + (size_t)(c == c0 ? slot0 : 2 * c) * stride; };
        float mm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, ll[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = c0; c <= c1; c += 8) {
          float v[8][4];
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[k][i] = c + k <= c1 && tok0 + (4 * ty + i) / hpc < w.s.n_new
                            ? __ldcg(reinterpret_cast<const float2*>(slot(c + k) + RF_ROWS * D) + 4 * ty + i).x
                            : -INFINITY;
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) mm[i] = fmaxf(mm[i], v[k][i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 4 * NC; ++c) o[i][c] = 0.f;
        for (int c = c0; c <= c1; c += 2) {
          float2 ml[2][4];
          float4 v[2][4][NC];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 4 * ty + i;
              const bool have = c + k <= c1 && tok0 + r / hpc < w.s.n_new;
              const float* pc = slot(have ? c + k : c0);
              ml[k][i] = have ? __ldcg(reinterpret_cast<const float2*>(pc + RF_ROWS * D) + r) : make_float2(-INFINITY, 0.f);
#pragma unroll
              for (int e = 0; e < NC; ++e)
                v[k][i][e] = have ? __ldcg(reinterpret_cast<const float4*>(pc + r * D + 64 * e + 4 * tx))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // no weight there. The maximum passes over NaN: a segment of NaN scores alone has
              // -inf and a sum of NaN, and counts.
              if (ml[k][i].x == -INFINITY && ml[k][i].y == 0.f) continue;
              const float f = exp2f(ml[k][i].x - mm[i]);
              ll[i] += ml[k][i].y * f;
#pragma unroll
              for (int e = 0; e < NC; ++e) {
                o[i][4 * e] += v[k][i][e].x * f;
                o[i][4 * e + 1] += v[k][i][e].y * f;
                o[i][4 * e + 2] += v[k][i][e].z * f;
                o[i][4 * e + 3] += v[k][i][e].w * f;
              }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) finish(i, ll[i]);
        if (tid == 0) counters[c0] = 0;  // re-armed for the next launch
      }
      __syncthreads();  // s_last is written again by the next cut segment
    }
  }
}

// ------------------------------------------------------------------ host side

size_t ragged_f32_ws_floats(int D) {
  return (size_t)2 * (RAGGED_F32_CTAS / 3 * (D == 64 ? 3 : 2)) * (RF_ROWS * D + 2 * RF_ROWS);
}

template <int D>
static cudaError_t ragged_f32(const RaggedAttnParams& p, float* part, int* counters, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  cudaError_t e = ensure_smem(attn_ragged_f32_kernel<D>, RfCfg<D>::SMEM, attr);
  if (e != cudaSuccess) return e;
  const int grid = std::min(num_sms, RAGGED_F32_CTAS / 3) * RfCfg<D>::PER_SM;
  attn_ragged_f32_kernel<D><<<grid, RF_THREADS, RfCfg<D>::SMEM, st>>>(p, part, counters,
                                                                      prefill_heads_per_cta(p.H / p.Hkv));
  return cudaGetLastError();
}

cudaError_t launch_attn_ragged_f32(const RaggedAttnParams& p, float* part, int* counters, int num_sms,
                                   cudaStream_t st) {
  return p.D == 128 ? ragged_f32<128>(p, part, counters, num_sms, st) : ragged_f32<64>(p, part, counters, num_sms, st);
}

}  // namespace llama
