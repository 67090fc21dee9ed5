// RoPE on packed q, k rows and the append of k, v to their pages.
//
// (x, y) -> (x cos - y sin, y cos + x sin) for the pairs (2i, 2i + 1) of each head of
// q and k, in fp32, rounded once; v is copied. Every value is read and written once,
// so the kernel is bound by HBM (large calls) or by its launch. A token's row belongs
// to 2^s threads of one block; a thread moves 8 consecutive values (16 or 32 bytes) at
// the same place of up to three heads, so its angles are read once, and issues all its
// loads before it waits for the first. 8 thousand tokens at 64/8 heads of 128 (bf16,
// 312 MB): 62 us, 5.0 TB/s (one thread per 8 values of the whole call: 86 us).
#include "kernels.cuh"

namespace llama {

namespace {
constexpr int RA_THREADS = 256;
constexpr int BATCH = 3;  // pieces a thread moves, at most (70B chunks: 2 61.6, 3 60.3, 4 66.5 us)
}

// 8 values as they lie in memory
template <typename TI> struct Raw8;
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <> struct Raw8<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_bf16x2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};

// 2^s threads a token (a multiple of D / 8)
template <typename TI, typename T, int D>
__global__ void __launch_bounds__(RA_THREADS) rope_append_kernel(const RopeAppendParams p, int s) {
  const int t = blockIdx.x * (RA_THREADS >> s) + (threadIdx.x >> s);
  if (t >= p.N) return;
  const int first = threadIdx.x & ((1 << s) - 1), d0 = first % (D / 8) * 8;
  const int slot = __ldg(p.slots + t), pos = __ldg(p.positions + t);
  if (slot == -1) return;
  const bool bad_pos = pos < 0 || pos >= p.n_pos, bad_slot = slot < 0 || slot >= (p.num_pages << p.page_shift);
  if (bad_pos || bad_slot) {
    if (first == 0 && blockIdx.y == 0) atomicOr(p.status, bad_pos ? LLAMA_DEV_POS_RANGE : LLAMA_DEV_PAGE_RANGE);
    return;
  }
  const float4* cs = reinterpret_cast<const float4*>(p.rope + (size_t)pos * (D / 2) + d0 / 2);
  const float4 a = __ldg(cs), b = __ldg(cs + 1);
  const float c[4] = {a.x, a.z, b.x, b.z}, n[4] = {a.y, a.w, b.y, b.w};
  const TI* row = reinterpret_cast<const TI*>(p.qkv) + (size_t)t * p.stride + d0;
  const size_t page = (size_t)(slot >> p.page_shift), off = slot & ((1 << p.page_shift) - 1);
  const int heads = p.H + 2 * p.Hkv, step = (1 << s) / (D / 8);
  const int h0 = first / (D / 8) + blockIdx.y * step, hop = step * gridDim.y;
  Raw8<TI> raw[BATCH];
#pragma unroll
  for (int i = 0; i < BATCH; ++i)
    if (h0 + i * hop < heads) raw[i].load(row + (size_t)(h0 + i * hop) * D);
#pragma unroll
  for (int i = 0; i < BATCH; ++i) {
    const int h = h0 + i * hop;
    if (h >= heads) break;
    float v[8];
    raw[i].get(v);
    if (h < p.H + p.Hkv) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = v[2 * k], y = v[2 * k + 1];
        v[2 * k] = x * c[k] - y * n[k];
        v[2 * k + 1] = y * c[k] + x * n[k];
      }
    }
    if (h < p.H) {
      store8(reinterpret_cast<T*>(p.q_out) + ((size_t)t * p.H + h) * D + d0, v);
    } else {
      const bool is_k = h < p.H + p.Hkv;
      const int kvh = h - p.H - (is_k ? 0 : p.Hkv);
      store8(reinterpret_cast<T*>(is_k ? p.k_pages : p.v_pages) + ((((page * p.Hkv + kvh) << p.page_shift) + off) * D + d0), v);
    }
  }
}

template <typename TI, typename T>
static cudaError_t rope_append(const RopeAppendParams& p, cudaStream_t st) {
  // as many threads as a row has pieces of 8 values, up to a block
  const int pieces = (p.H + 2 * p.Hkv) * p.D / 8;
  int s = 5;
  while ((1 << s) < pieces && (1 << s) < RA_THREADS) ++s;
  const int per = RA_THREADS >> s;
  // so many blocks for a row that a thread has at most BATCH pieces, all in flight at once
  const int each = (pieces + (1 << s) - 1) >> s, split = (each + BATCH - 1) / BATCH;
  const dim3 grid((unsigned)((p.N + (long long)per - 1) / per), split);
  if (split > 65535) return cudaErrorInvalidValue;
  if (p.D == 128)
    rope_append_kernel<TI, T, 128><<<grid, RA_THREADS, 0, st>>>(p, s);
  else
    rope_append_kernel<TI, T, 64><<<grid, RA_THREADS, 0, st>>>(p, s);
  return cudaGetLastError();
}

cudaError_t launch_rope_append(const RopeAppendParams& p, bool in_bf16, bool out_bf16, cudaStream_t st) {
  if (in_bf16) return rope_append<bf16, bf16>(p, st);
  return out_bf16 ? rope_append<float, bf16>(p, st) : rope_append<float, float>(p, st);
}

}  // namespace llama
