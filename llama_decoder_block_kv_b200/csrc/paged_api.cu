// C entry points of the serving operators over a paged cache: argument checks
// on the host, then one launch each on the caller's stream and current device.
#include "kernels.cuh"

#include <algorithm>

using namespace llama;

namespace {

bool aligned(const void* p, size_t a = 16) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

bool heads_ok(int dtype, int H, int Hkv, int D) {
  return (dtype == LLAMA_FP32 || dtype == LLAMA_BF16) && H >= 1 && Hkv >= 1 && H % Hkv == 0 && H <= (1 << 16) &&
         (D == 64 || D == 128);
}

// Keys of a request and tokens of a call: the kernels' tiles and units go past them by up to 255 in 32 bits
constexpr long long MAX_LEN = (1LL << 31) - 256;

bool pool_ok(const llama_page_args* a) {
  return a && page_shift(a->page_size) > 0 && a->num_pages >= 1 && a->max_pages >= 1 &&
         (long long)a->max_pages * a->page_size <= MAX_LEN && (long long)a->num_pages * a->page_size < (1LL << 31);
}

bool stride_ok(int64_t stride, int64_t width, int esz) {
  return stride >= width && stride * esz % 16 == 0 && stride < (1LL << 31);
}

int launched(cudaError_t e) { return e == cudaSuccess ? LLAMA_OK : LLAMA_ERR_CUDA; }

// SMs of the current device (asked once per device)
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// the flags that a status call has returned, and no others: more may be raised meanwhile
__global__ void clear_flags_kernel(int* status, int flags) { atomicAnd(status, ~flags); }

}  // namespace

namespace llama {

int page_shift(int ps) { return ps == 16 ? 4 : ps == 32 ? 5 : ps == 64 ? 6 : ps == 128 ? 7 : -1; }

bool page_args_ok(const llama_page_args* a) {
  return pool_ok(a) && heads_ok(a->dtype, a->n_heads, a->n_kv_heads, a->head_dim) &&
         (long long)a->num_pages * a->n_kv_heads * a->page_size < (1LL << 31);
}

// Workspace: counters, then partials.
static constexpr size_t WS_COUNTERS = 4096;
static_assert((RAGGED_TC_CTAS + RAGGED_DECODE_CTAS) * sizeof(int) <= WS_COUNTERS && RAGGED_F32_CTAS * sizeof(int) <= WS_COUNTERS,
              "counters");

size_t ragged_ws_bytes(int dtype, int D) {
  return WS_COUNTERS +
         sizeof(float) * (dtype == LLAMA_BF16 ? std::max(ragged_tc_ws_floats(D), ragged_decode_ws_floats(D)) : ragged_f32_ws_floats(D));
}

int ragged_attention(const RaggedAttnParams& p, int dtype, void* workspace, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return LLAMA_ERR_CUDA;
  int* counters = static_cast<int*>(workspace);
  float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + WS_COUNTERS);
  if (dtype == LLAMA_BF16 && p.tables && p.max_new == 1)
    return launched(launch_attn_ragged_decode(p, part, counters + RAGGED_TC_CTAS, sms, st));
  if (dtype == LLAMA_BF16) return launched(launch_attn_ragged_tc(p, part, counters, sms, st));
  return launched(launch_attn_ragged_f32(p, part, counters, sms, st));
}

}  // namespace llama

extern "C" {

int llama_page_plan(const llama_page_args* a, const int32_t* cached, const int32_t* fresh, int n_seqs, int max_tokens,
                    int32_t* tables, int32_t* free_pages, const int32_t* free_count, int32_t* free_count_out,
                    int32_t* cu, int32_t* kv_lens, int32_t* positions, int32_t* slots, int32_t* status, void* stream) {
  if (!pool_ok(a) || n_seqs < 1 || n_seqs > LLAMA_MAX_SEQS || max_tokens < 1) return LLAMA_ERR_INVALID_ARGS;
  if (!aligned(cached, 4) || !aligned(fresh, 4) || !aligned(tables, 4) || !aligned(free_pages, 4) ||
      !aligned(free_count, 4) || !aligned(free_count_out, 4) || !aligned(cu, 4) || !aligned(kv_lens, 4) ||
      !aligned(positions) || !aligned(slots) || !aligned(status, 4))
    return LLAMA_ERR_INVALID_ARGS;
  PagePlanParams p = {};
  p.cached = cached;
  p.fresh = fresh;
  p.B = n_seqs;
  p.max_tokens = max_tokens;
  p.page_shift = page_shift(a->page_size);
  p.num_pages = a->num_pages;
  p.max_pages = a->max_pages;
  p.tables = tables;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.free_count_out = free_count_out;
  p.cu = cu;
  p.kv_lens = kv_lens;
  p.positions = positions;
  p.slots = slots;
  p.status = status;
  return launched(launch_page_plan(p, reinterpret_cast<cudaStream_t>(stream)));
}

int llama_rope_append(const llama_page_args* a, const void* qkv, int64_t qkv_stride, int qkv_dtype,
                      const int32_t* positions, const int32_t* slots, int n_tokens, const float* rope, int n_pos,
                      void* q_out, void* k_pages, void* v_pages, int32_t* status, void* stream) {
  if (!page_args_ok(a) || n_tokens < 1 || n_pos < 1) return LLAMA_ERR_INVALID_ARGS;
  if (qkv_dtype != LLAMA_FP32 && (qkv_dtype != LLAMA_BF16 || a->dtype != LLAMA_BF16)) return LLAMA_ERR_INVALID_ARGS;
  const int64_t width = (int64_t)(a->n_heads + 2 * a->n_kv_heads) * a->head_dim;
  if (!stride_ok(qkv_stride, width, qkv_dtype == LLAMA_BF16 ? 2 : 4)) return LLAMA_ERR_INVALID_ARGS;
  if (!aligned(qkv) || !aligned(positions, 4) || !aligned(slots, 4) || !aligned(rope) || !aligned(q_out) ||
      !aligned(k_pages) || !aligned(v_pages) || !aligned(status, 4))
    return LLAMA_ERR_INVALID_ARGS;
  RopeAppendParams p = {};
  p.qkv = qkv;
  p.stride = qkv_stride;
  p.positions = positions;
  p.slots = slots;
  p.N = n_tokens;
  p.H = a->n_heads;
  p.Hkv = a->n_kv_heads;
  p.D = a->head_dim;
  p.page_shift = page_shift(a->page_size);
  p.num_pages = a->num_pages;
  p.n_pos = n_pos;
  p.rope = reinterpret_cast<const float2*>(rope);
  p.q_out = q_out;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.status = status;
  return launched(launch_rope_append(p, qkv_dtype == LLAMA_BF16, a->dtype == LLAMA_BF16,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

int64_t llama_attn_workspace_bytes(int dtype, int n_heads, int n_kv_heads, int head_dim) {
  if (!heads_ok(dtype, n_heads, n_kv_heads, head_dim)) return LLAMA_ERR_INVALID_ARGS;
  return (int64_t)ragged_ws_bytes(dtype, head_dim);
}

int llama_attn_paged(const llama_page_args* a, const void* q, int64_t q_stride, const void* k_pages,
                     const void* v_pages, const int32_t* tables, const int32_t* cu, const int32_t* kv_lens, int n_seqs,
                     int n_tokens, int max_new, void* out, void* workspace, int64_t workspace_bytes, int32_t* status,
                     void* stream) {
  if (!page_args_ok(a) || n_seqs < 1 || n_seqs > LLAMA_MAX_SEQS || n_tokens < 1 || n_tokens > MAX_LEN || max_new < 1)
    return LLAMA_ERR_INVALID_ARGS;
  if (!stride_ok(q_stride, (int64_t)a->n_heads * a->head_dim, a->dtype == LLAMA_BF16 ? 2 : 4))
    return LLAMA_ERR_INVALID_ARGS;
  if (!aligned(q) || !aligned(k_pages) || !aligned(v_pages) || !aligned(tables, 4) || !aligned(cu, 4) ||
      !aligned(kv_lens, 4) || !aligned(out) || !aligned(workspace, 256) || !aligned(status, 4) ||
      workspace_bytes < llama_attn_workspace_bytes(a->dtype, a->n_heads, a->n_kv_heads, a->head_dim))
    return LLAMA_ERR_INVALID_ARGS;
  RaggedAttnParams p = {};
  p.q = q;
  p.q_stride = q_stride;
  p.k = k_pages;
  p.v = v_pages;
  p.tables = tables;
  p.cu = cu;
  p.kv_lens = kv_lens;
  p.B = n_seqs;
  p.N = n_tokens;
  p.max_new = std::min(max_new, n_tokens);
  p.H = a->n_heads;
  p.Hkv = a->n_kv_heads;
  p.D = a->head_dim;
  p.page_shift = page_shift(a->page_size);
  p.num_pages = a->num_pages;
  p.max_pages = a->max_pages;
  p.o = out;
  p.status = status;
  return ragged_attention(p, a->dtype, workspace, reinterpret_cast<cudaStream_t>(stream));
}

int llama_attn_packed(int dtype, int n_heads, int n_kv_heads, int head_dim, const void* q, int64_t q_stride,
                      const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int32_t* cu, int n_seqs,
                      int n_tokens, int max_len, void* out, void* workspace, int64_t workspace_bytes, int32_t* status,
                      void* stream) {
  if (!heads_ok(dtype, n_heads, n_kv_heads, head_dim) || n_seqs < 1 || n_seqs > LLAMA_MAX_SEQS || n_tokens < 1 ||
      n_tokens > MAX_LEN || max_len < 1)
    return LLAMA_ERR_INVALID_ARGS;
  const int esz = dtype == LLAMA_BF16 ? 2 : 4;
  const int64_t kw = (int64_t)n_kv_heads * head_dim;
  if (!stride_ok(q_stride, (int64_t)n_heads * head_dim, esz) || !stride_ok(k_stride, kw, esz) ||
      !stride_ok(v_stride, kw, esz))
    return LLAMA_ERR_INVALID_ARGS;
  if (!aligned(q) || !aligned(k) || !aligned(v) || !aligned(cu, 4) || !aligned(out) || !aligned(workspace, 256) ||
      !aligned(status, 4) || workspace_bytes < llama_attn_workspace_bytes(dtype, n_heads, n_kv_heads, head_dim))
    return LLAMA_ERR_INVALID_ARGS;
  RaggedAttnParams p = {};
  p.q = q;
  p.q_stride = q_stride;
  p.k = k;
  p.k_stride = k_stride;
  p.v = v;
  p.v_stride = v_stride;
  p.cu = cu;
  p.B = n_seqs;
  p.N = n_tokens;
  p.max_new = std::min(max_len, n_tokens);
  p.H = n_heads;
  p.Hkv = n_kv_heads;
  p.D = head_dim;
  p.o = out;
  p.status = status;
  return ragged_attention(p, dtype, workspace, reinterpret_cast<cudaStream_t>(stream));
}

int llama_paged_status(int32_t* status, int* flags) {
  if (flags) *flags = 0;
  if (!status) return LLAMA_ERR_INVALID_ARGS;
  cudaPointerAttributes at;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaPointerGetAttributes(&at, status) != cudaSuccess) return LLAMA_ERR_CUDA;
  if (at.type == cudaMemoryTypeUnregistered || (at.type == cudaMemoryTypeDevice && at.device != dev)) return LLAMA_ERR_INVALID_ARGS;
  int w = 0;
  if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpy(&w, status, sizeof(int), cudaMemcpyDefault) != cudaSuccess)
    return LLAMA_ERR_CUDA;
  if (w) {
    // done before this returns: streams that do not wait for the default one may raise flags right after
    clear_flags_kernel<<<1, 1>>>(status, w);
    if (cudaGetLastError() != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess) return LLAMA_ERR_CUDA;
  }
  if (flags) *flags = w;
  if (w & LLAMA_DEV_TIMEOUT) return LLAMA_ERR_TIMEOUT;
  if (w & LLAMA_DEV_PAGE_RANGE) return LLAMA_ERR_PAGE_RANGE;
  if (w & LLAMA_DEV_OUT_OF_PAGES) return LLAMA_ERR_OUT_OF_PAGES;
  if (w & LLAMA_DEV_POS_RANGE) return LLAMA_ERR_POS_RANGE;
  return LLAMA_OK;
}

}  // extern "C"
