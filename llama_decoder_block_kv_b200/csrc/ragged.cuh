// Device parts shared by the attention kernels of packed rows: a request's
// lengths with their checks, and one row computed by a warp, key by key.
#pragma once

#include "kernels.cuh"

namespace llama {

// Request b's new tokens and keys, from device memory, with the checks of the
// header: false (and the position range flag) for a request that is skipped.
struct RaggedSeq {
  int q0, n_new, kv;  // first row, new tokens, keys
};
__device__ __forceinline__ bool ragged_seq(const RaggedAttnParams& p, int b, RaggedSeq& s, bool flag) {
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
    if (flag) atomicOr(p.status, LLAMA_DEV_POS_RANGE);
  }
  return ok;
}


// Row tok of the request, query head h, by one warp: softmax(q.k / sqrt(D)) V
// with a running maximum and sum in fp32, the head dimension over the lanes.
template <typename T, int D>
__device__ void ragged_row(const RaggedAttnParams& p, int b, const RaggedSeq& s, int tok, int h, int lane) {
  constexpr int E = D / 32;
  const int kvh = h / (p.H / p.Hkv);
  const int n = min(s.kv - s.n_new + tok + 1, s.kv);
  const float scale = rsqrtf((float)D);
  const size_t row = (size_t)(s.q0 + tok);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_f32(reinterpret_cast<const T*>(p.q)[row * p.q_stride + h * D + e * 32 + lane]);
    o[e] = 0.f;
  }
  for (int j = 0; j < n; ++j) {
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
    float dot = 0.f, vf[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float kf = have ? to_f32(reinterpret_cast<const T*>(p.k)[ka + e * 32 + lane]) : 0.f;
      vf[e] = have ? to_f32(reinterpret_cast<const T*>(p.v)[va + e * 32 + lane]) : 0.f;
      dot += q[e] * kf;
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
    reinterpret_cast<T*>(p.o)[(row * p.H + h) * D + e * 32 + lane] = from_f32<T>(n > 0 ? o[e] / l : 0.f);
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
