// What the queries of an absorbed latent attention looked at, per cached token.
#include <cmath>

#include "kv_fp4.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int kWThreads = 256;

struct WeightParams {
  KvView kv;
  int layer, B, Q, heads, fp4;
  float scale_log2, decay;
  const __nv_bfloat16* q;
  const int32_t* seqs;
  const float* lse;
  float* weights;
  uint32_t* status;
};

// A warp a token: its row in shared memory, then one query row after the other.
__global__ void __launch_bounds__(kWThreads) weights_kernel(const WeightParams p) {
  extern __shared__ __nv_bfloat16 rows[];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seq = p.seqs[b];
  bool good = seq >= 0 && seq < p.kv.max_seqs;
  for (int j = 0; good && j < b; ++j) good = p.seqs[j] != seq;
  if (!good) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, MOE_DEV_ERR_BAD_SEQ);
    return;
  }
  const int len = p.kv.len_of(seq), dim = p.kv.rank + p.kv.rope;
  __nv_bfloat16* row = rows + warp * dim;
  const size_t cap = (size_t)p.kv.max_blocks << p.kv.page_shift;
  for (int t = blockIdx.x * (kWThreads / 32) + warp; t < len; t += gridDim.x * (kWThreads / 32)) {
    int pg = p.kv.table[(size_t)seq * p.kv.max_blocks + (t >> p.kv.page_shift)];
    if (pg < 0 || pg >= p.kv.n_pages) {
      set_status(p.status, MOE_DEV_ERR_BAD_PAGE);
      pg = 0;
    }
    const __nv_bfloat16* src = p.kv.pages + p.kv.row_offset(p.layer, pg, t & (p.kv.page_tokens - 1));
    __syncwarp();
    for (int d = lane; d < dim; d += 32) {
      if (d >= p.kv.rank) row[d] = src[p.kv.rope_at + d - p.kv.rank];
      else if (!p.fp4) row[d] = src[d];
      else {
        const uint8_t* bytes = reinterpret_cast<const uint8_t*>(src);
        const uint32_t c = bytes[d / 2] >> (d & 1 ? 4 : 0) & 15;
        const uint4 v = fp4_expand8(c, fp4_factor(bytes[p.kv.rank / 2 + 2 * p.kv.rope + d / kFpBlock]));
        row[d] = __ushort_as_bfloat16((unsigned short)(v.x & 0xFFFFu));
      }
    }
    __syncwarp();
    float sum = 0.0f;
    for (int r = 0; r < p.Q * p.heads; ++r) {
      if (t >= len - p.Q + r / p.heads + 1) continue;
      const size_t at = (size_t)b * p.Q * p.heads + r;
      float s = 0.0f;
      for (int d = lane; d < dim; d += 32) s = fmaf(__bfloat162float(p.q[at * dim + d]), __bfloat162float(row[d]), s);
      s = warp_sum(s);
      sum += tc::ex2(fmaf(s, p.scale_log2, -p.lse[at] * 1.4426950408889634f));
    }
    if (lane == 0) {
      float* w = p.weights + (size_t)seq * cap + t;
      *w = p.decay == 0.0f ? sum : fmaf(p.decay, *w, sum);
    }
  }
}

bool weights_shape_ok(int B, int Q, int heads) { return B <= 4096 && (long long)Q * heads <= 1024; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_latent_weights_workspace_size(const moe_kv_cache* cache, int B, int Q, int heads) {
  if (check_latent(cache, 0) != MOE_OK || B < 1 || Q < 1 || heads < 1 || !weights_shape_ok(B, Q, heads)) return 0;
  return 256;
}

int moe_latent_weights(const moe_kv_cache* cache, int layer, const void* q, const int32_t* seqs, int B, int Q, int heads,
                       float scale, const float* lse, float decay, float* weights, void* ws, size_t ws_bytes,
                       uint32_t* dev_status, moe_stream_t stream) {
  int st = check_latent(cache, layer);
  if (st == MOE_ERR_INVALID_ARG || check_kv(cache) != MOE_OK) return st;
  if (B < 0 || Q < 1 || heads < 1 || !std::isfinite(scale) || !(decay >= 0.0f && decay <= 1.0f)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && (!q || !seqs || !lse || !weights)) return MOE_ERR_INVALID_ARG;
  if (st != MOE_OK) return st;
  if (!weights_shape_ok(B, Q, heads)) return MOE_ERR_UNSUPPORTED;
  if (B == 0) return MOE_OK;
  if (!kv_aligned(q, 16) || !kv_aligned(lse, 4) || !kv_aligned(weights, 4)) return MOE_ERR_UNSUPPORTED;
  st = check_ws(ws, ws_bytes, moe_latent_weights_workspace_size(cache, B, Q, heads));
  if (st != MOE_OK) return st;
  WeightParams p;
  p.kv = kv_view(*cache);
  p.layer = layer;
  p.B = B;
  p.Q = Q;
  p.heads = heads;
  p.fp4 = cache->format == MOE_KV_FP4;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.decay = decay;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.seqs = seqs;
  p.lse = lse;
  p.weights = weights;
  p.status = dev_status;
  const size_t smem = (size_t)(kWThreads / 32) * (cache->rank + cache->rope) * 2;
  const int per = 8 * num_sms() / B + 1;
  return launch_k(weights_kernel, dim3(per, B), kWThreads, smem, reinterpret_cast<cudaStream_t>(stream), p) == cudaSuccess
             ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
