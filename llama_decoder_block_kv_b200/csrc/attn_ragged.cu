// Causal attention of packed rows over a paged cache or over packed keys, one
// warp per (row, query head): softmax(q.k / sqrt(D)) V with a running maximum
// and sum in fp32, keys in turn, the head dimension over the lanes.
#include "kernels.cuh"

namespace llama {

namespace {
constexpr int AR_WARPS = 4;
}

template <typename T, int D>
__global__ void __launch_bounds__(AR_WARPS * 32) attn_ragged_rows_kernel(const RaggedAttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long it = (long long)blockIdx.x * AR_WARPS + (threadIdx.x >> 5);
  const int t = (int)(it / p.H), h = (int)(it - (long long)t * p.H);
  // requests in turn: a malformed cu must not mislead a bisection
  if (t >= p.N) return;
  RaggedSeq s;
  int b = 0;
  for (; b < p.B; ++b)
    if (ragged_seq(p, b, s, t == 0 && h == 0 && lane == 0) && t >= s.q0 && t < s.q0 + s.n_new) break;
  if (b == p.B) return;
  if (t == 0 && h == 0 && lane == 0)
    for (int c = b + 1; c < p.B; ++c) {
      RaggedSeq u;
      ragged_seq(p, c, u, true);
    }
  const int kvh = h / (p.H / p.Hkv);
  const int pos = s.kv - s.n_new + t - s.q0, n = min(pos + 1, s.kv);
  const float scale = rsqrtf((float)D);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_f32(reinterpret_cast<const T*>(p.q)[(size_t)t * p.q_stride + h * D + e * 32 + lane]);
    o[e] = 0.f;
  }
  for (int j = 0; j < n; ++j) {
    float kf[E], vf[E];
    bool have = true;
    size_t ka, va;
    if (p.tables) {
      const int page = p.tables[(size_t)b * p.max_pages + (j >> p.page_shift)];
      have = (unsigned)page < (unsigned)p.num_pages;
      if (!have && lane == 0) atomicOr(p.status, LLAMA_DEV_PAGE_RANGE);
      ka = va = (((((size_t)page * p.Hkv + kvh) << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * D);
    } else {
      ka = (size_t)(s.q0 + j) * p.k_stride + kvh * D;
      va = (size_t)(s.q0 + j) * p.v_stride + kvh * D;
    }
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      kf[e] = have ? to_f32(reinterpret_cast<const T*>(p.k)[ka + e * 32 + lane]) : 0.f;
      vf[e] = have ? to_f32(reinterpret_cast<const T*>(p.v)[va + e * 32 + lane]) : 0.f;
      dot += q[e] * kf[e];
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
    dot *= scale;
    const float mn = fmaxf(m, dot);
    const float a = m == -INFINITY ? 0.f : expf(m - mn), w = expf(dot - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * vf[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    reinterpret_cast<T*>(p.o)[((size_t)t * p.H + h) * D + e * 32 + lane] = from_f32<T>(n > 0 ? o[e] / l : 0.f);
}

template <typename T>
cudaError_t launch_attn_ragged_rows(const RaggedAttnParams& p, cudaStream_t st) {
  const long long items = (long long)p.N * p.H;
  const unsigned grid = (unsigned)((items + AR_WARPS - 1) / AR_WARPS);
  if (p.D == 128)
    attn_ragged_rows_kernel<T, 128><<<grid, AR_WARPS * 32, 0, st>>>(p);
  else
    attn_ragged_rows_kernel<T, 64><<<grid, AR_WARPS * 32, 0, st>>>(p);
  return cudaGetLastError();
}

template cudaError_t launch_attn_ragged_rows<float>(const RaggedAttnParams&, cudaStream_t);
template cudaError_t launch_attn_ragged_rows<bf16>(const RaggedAttnParams&, cudaStream_t);

}  // namespace llama
