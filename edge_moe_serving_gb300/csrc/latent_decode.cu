// Absorbed latent attention over the paged cache: every head's keys are the
// cached rows themselves and its values their first `rank` entries.
//
// Simple form: one CTA per (query token, head).  Its warps take the tokens in
// turn; a warp holds the query and its running output in registers, 32 lanes
// over the row, and keeps the running maximum m and sum l of the softmax
// (log2 domain), so each row is read once: o and l are scaled by 2^(m - m')
// when the maximum grows.  The warps' (m, l, o) are joined at the end.
#include <cmath>

#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxRow = 576;

struct DecodeParams {
  KvView kv;
  int layer, B, Q, heads, shared;
  float scale_log2;   // scale * log2(e): the exponentials are powers of two
  const __nv_bfloat16* q;
  const int32_t* seqs;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
};

__global__ void __launch_bounds__(32 * kWarps)
decode_simple_kernel(const DecodeParams p) {
  __shared__ float s_o[kWarps][512];
  __shared__ float s_m[kWarps], s_l[kWarps];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = p.kv.row, rank = p.kv.rank;
  const size_t qrow = blockIdx.x;   // (b*Q + i)*heads + h
  const int bq = (int)(qrow / p.heads), b = bq / p.Q, i = bq - b * p.Q;
  const int seq = p.seqs[b], prefix_seq = p.seqs[0];
  const bool good = seq >= 0 && seq < p.kv.max_seqs && prefix_seq >= 0 && prefix_seq < p.kv.max_seqs;
  if (!good && threadIdx.x == 0) set_status(p.status, MOE_DEV_ERR_BAD_SEQ);
  const int limit = good ? p.kv.len_of(seq) - p.Q + i + 1 : 0;
  float q[kMaxRow / 32], o[512 / 32];
#pragma unroll
  for (int j = 0; j < kMaxRow / 32; ++j) {
    const int d = lane + 32 * j;
    q[j] = d < row ? __bfloat162float(p.q[qrow * row + d]) : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 512 / 32; ++j) o[j] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  for (int t = warp; t < limit; t += kWarps) {
    const int s = t < p.shared ? prefix_seq : seq;
    int page = p.kv.table[(size_t)s * p.kv.max_blocks + (t >> p.kv.page_shift)];
    if (page < 0 || page >= p.kv.n_pages) {
      if (lane == 0) set_status(p.status, MOE_DEV_ERR_BAD_PAGE);
      page = 0;
    }
    const __nv_bfloat16* k = p.kv.pages + p.kv.row_offset(p.layer, page, t & (p.kv.page_tokens - 1));
    float x[kMaxRow / 32], dot = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxRow / 32; ++j) {
      const int d = lane + 32 * j;
      x[j] = d < row ? __bfloat162float(k[d]) : 0.0f;
      dot = fmaf(q[j], x[j], dot);
    }
    const float s2 = warp_sum(dot) * p.scale_log2;
    const float mn = fmaxf(m, s2);
    const float ref = mn == -INFINITY ? 0.0f : mn;
    const float f = exp2f(m - ref), w = exp2f(s2 - ref);
    l = fmaf(l, f, w);
#pragma unroll
    for (int j = 0; j < 512 / 32; ++j) o[j] = fmaf(w, x[j], o[j] * f);
    m = mn;
  }
#pragma unroll
  for (int j = 0; j < 512 / 32; ++j) s_o[warp][lane + 32 * j] = o[j];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  const float ref = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  for (int w = 0; w < kWarps; ++w) sum = fmaf(s_l[w], exp2f(s_m[w] - ref), sum);
  for (int d = threadIdx.x; d < rank; d += blockDim.x) {
    float v = 0.0f;
    for (int w = 0; w < kWarps; ++w) v = fmaf(s_o[w][d], exp2f(s_m[w] - ref), v);
    p.out[qrow * rank + d] = __float2bfloat16_rn(limit > 0 ? v / sum : 0.0f);
  }
  if (p.lse && threadIdx.x == 0) p.lse[qrow] = limit > 0 ? (ref + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_latent_decode_workspace_size(const moe_kv_cache* cache, int B, int Q, int heads, int shared_tokens) {
  (void)cache, (void)B, (void)Q, (void)heads, (void)shared_tokens;
  return 0;
}

int moe_latent_decode(const moe_kv_cache* cache, int layer, const void* q, const int32_t* seqs, int B, int Q,
                      int heads, float scale, int shared_tokens, void* out, float* lse_opt, void* ws, size_t ws_bytes,
                      uint32_t* dev_status, moe_stream_t stream) {
  const int st = check_latent(cache, layer);
  if (st == MOE_ERR_INVALID_ARG || check_kv(cache) != MOE_OK) return st;
  if (B < 0 || Q < 1 || heads < 1 || shared_tokens < 0 || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (shared_tokens % cache->page_tokens || shared_tokens / cache->page_tokens > cache->max_blocks)
    return MOE_ERR_INVALID_ARG;
  if (B > 0 && (!q || !seqs || !out)) return MOE_ERR_INVALID_ARG;
  if (st != MOE_OK) return st;
  if (B > 4096 || (long long)Q * heads > 1024) return MOE_ERR_UNSUPPORTED;
  if (B == 0) return MOE_OK;
  if (!kv_aligned(q, 16) || !kv_aligned(out, 16)) return MOE_ERR_UNSUPPORTED;
  (void)ws, (void)ws_bytes;
  DecodeParams p;
  p.kv = kv_view(*cache);
  p.layer = layer;
  p.B = B;
  p.Q = Q;
  p.heads = heads;
  p.shared = shared_tokens;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.seqs = seqs;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse_opt;
  p.status = dev_status;
  const cudaError_t e = launch_k(decode_simple_kernel, B * Q * heads, 32 * kWarps, 0,
                                 reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
