// Causal attention of packed rows over a paged cache or over packed keys, one
// warp per (row, query head): softmax(q.k / sqrt(D)) V with a running maximum
// and sum in fp32, keys in turn, the head dimension over the lanes.
#include "ragged.cuh"

namespace llama {

namespace {
constexpr int AR_WARPS = 4;
}

template <typename T, int D>
__global__ void __launch_bounds__(AR_WARPS * 32) attn_ragged_rows_kernel(const RaggedAttnParams p) {
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
  ragged_row<T, D>(p, b, s, t - s.q0, h, lane);
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
