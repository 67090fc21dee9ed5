// RoPE on packed q, k rows and the append of k, v to their pages.
//
// (x, y) -> (x cos - y sin, y cos + x sin) for the pairs (2i, 2i + 1) of each
// head of q and k, in fp32, rounded once; v is copied. Every value is read and
// written once, so the kernel is bound by HBM (large calls) or by its launch.
// A thread moves 8 consecutive values (16 or 32 bytes) of one row.
#include "kernels.cuh"

#include <algorithm>

namespace llama {

namespace {
constexpr int RA_THREADS = 256;
}

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float* v) {
  const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <typename TI, typename T>
__global__ void __launch_bounds__(RA_THREADS) rope_append_kernel(const RopeAppendParams p) {
  const int D = p.D, HD = p.H * D, KD = p.Hkv * D, chunks = (HD + 2 * KD) / 8;
  const long long items = (long long)p.N * chunks;
  for (long long it = (long long)blockIdx.x * RA_THREADS + threadIdx.x; it < items;
       it += (long long)gridDim.x * RA_THREADS) {
    const int t = (int)(it / chunks), n0 = (int)(it - (long long)t * chunks) * 8;
    const int slot = p.slots[t], pos = p.positions[t];
    if (slot == -1) continue;
    if (pos < 0 || pos >= p.n_pos) {
      atomicOr(p.status, LLAMA_DEV_POS_RANGE);
      continue;
    }
    if (slot < 0 || slot >= (p.num_pages << p.page_shift)) {
      atomicOr(p.status, LLAMA_DEV_PAGE_RANGE);
      continue;
    }
    float v[8];
    load8(reinterpret_cast<const TI*>(p.qkv) + (size_t)t * p.stride + n0, v);
    const int d0 = n0 % D;
    if (n0 < HD + KD) {
      const float4* cs = reinterpret_cast<const float4*>(p.rope + (size_t)pos * (D / 2) + d0 / 2);
      const float4 c0 = cs[0], c1 = cs[1];
      const float c[4] = {c0.x, c0.z, c1.x, c1.z}, s[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = v[2 * i], y = v[2 * i + 1];
        v[2 * i] = x * c[i] - y * s[i];
        v[2 * i + 1] = y * c[i] + x * s[i];
      }
    }
    if (n0 < HD) {
      store8(reinterpret_cast<T*>(p.q_out) + (size_t)t * HD + n0, v);
    } else {
      const bool is_k = n0 < HD + KD;
      const int kvh = (n0 - HD - (is_k ? 0 : KD)) / D;
      const size_t page = (size_t)(slot >> p.page_shift), off = slot & ((1 << p.page_shift) - 1);
      store8(reinterpret_cast<T*>(is_k ? p.k_pages : p.v_pages) +
                 ((((page * p.Hkv + kvh) << p.page_shift) + off) * D + d0),
             v);
    }
  }
}

cudaError_t launch_rope_append(const RopeAppendParams& p, bool in_bf16, bool out_bf16, cudaStream_t st) {
  const long long items = (long long)p.N * ((p.H + 2 * p.Hkv) * p.D / 8);
  const unsigned grid = (unsigned)std::min<long long>((items + RA_THREADS - 1) / RA_THREADS, 1 << 16);
  if (in_bf16)
    rope_append_kernel<bf16, bf16><<<grid, RA_THREADS, 0, st>>>(p);
  else if (out_bf16)
    rope_append_kernel<float, bf16><<<grid, RA_THREADS, 0, st>>>(p);
  else
    rope_append_kernel<float, float><<<grid, RA_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace llama
