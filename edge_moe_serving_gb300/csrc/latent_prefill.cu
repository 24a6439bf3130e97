// Expanded latent attention of prompt tokens: keys and values are made per
// head from the cached latents, then a causal softmax attention reads them.
//
// Simple form.  expand_kernel: k and v of every cached token and head into the
// workspace, 32 x 32 output tiles over 32-wide slices of the latents in shared
// memory (fp32 sums, rounded to bf16 once).  attend_kernel: one warp per
// (query row, head) with the query and the running output in registers and
// the softmax's running maximum and sum, each key and value read once per
// row.
#include <cmath>

#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kTile = 32;
constexpr int kRowAlign = 128;   // sequences start at multiples of this in the expanded buffers

struct PrefillParams {
  KvView kv;
  int layer, B, T, heads, dn, dv, kv_rows;
  float scale_log2;
  const __nv_bfloat16* q;
  const int32_t* seqs;
  const int32_t* q_off;
  const __nv_bfloat16* w;
  __nv_bfloat16* out;
  int32_t* base;            // [B + 1] first expanded row of each sequence; base[B] < 0: over capacity
  __nv_bfloat16* k;         // [heads, kv_rows, dn]
  __nv_bfloat16* v;         // [heads, kv_rows, dv]
  uint32_t* status;
};

__device__ inline int seq_len(const PrefillParams& p, int b) {
  const int s = p.seqs[b];
  return s >= 0 && s < p.kv.max_seqs ? p.kv.len_of(s) : 0;
}

// One CTA: where each sequence's expanded rows begin.
__global__ void layout_kernel(const PrefillParams p) {
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x != 0) return;
  long long at = 0;
  for (int b = 0; b < p.B; ++b) {
    p.base[b] = (int)at;
    at += (seq_len(p, b) + kRowAlign - 1) / kRowAlign * kRowAlign;
    if (at > p.kv_rows) {
      p.base[p.B] = -1;
      set_status(p.status, MOE_DEV_ERR_CAPACITY);
      return;
    }
  }
  p.base[p.B] = (int)at;
}

__global__ void __launch_bounds__(kTile * kTile / 4) expand_kernel(const PrefillParams p) {
  __shared__ float sx[kTile][kTile + 1], sw[kTile][kTile + 1];
  pdl_wait();
  pdl_trigger();
  const int total = p.base[p.B];
  const int r0 = blockIdx.x * kTile;
  if (r0 >= total) return;
  int b = 0;
  while (b + 1 < p.B && p.base[b + 1] <= r0) ++b;
  const int t0 = r0 - p.base[b], len = seq_len(p, b);
  if (t0 >= len) return;
  const int feats = p.dn + p.dv;
  const int f0 = blockIdx.y * kTile;   // feature of all heads: a tile lies in one head's keys or values
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float acc[4] = {};
  for (int c0 = 0; c0 < p.kv.rank; c0 += kTile) {
    for (int j = ty; j < kTile; j += 8) {
      const int t = t0 + j;
      float x = 0.0f;
      if (t < len) {
        int page = p.kv.table[(size_t)p.seqs[b] * p.kv.max_blocks + (t >> p.kv.page_shift)];
        if (page < 0 || page >= p.kv.n_pages) {
          if (tx == 0) set_status(p.status, MOE_DEV_ERR_BAD_PAGE);
          page = 0;
        }
        x = __bfloat162float(p.kv.pages[p.kv.row_offset(p.layer, page, t & (p.kv.page_tokens - 1)) + c0 + tx]);
      }
      sx[j][tx] = x;
      sw[j][tx] = __bfloat162float(p.w[(size_t)(f0 + j) * p.kv.rank + c0 + tx]);
    }
    __syncthreads();
    for (int c = 0; c < kTile; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = fmaf(sx[ty + 8 * j][c], sw[tx][c], acc[j]);
    __syncthreads();
  }
  const int h = f0 / feats, f = f0 - h * feats + tx;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (t0 + ty + 8 * j >= len) continue;
    const size_t r = (size_t)h * p.kv_rows + r0 + ty + 8 * j;
    if (f < p.dn) p.k[r * p.dn + f] = __float2bfloat16_rn(acc[j]);
    else p.v[r * p.dv + f - p.dn] = __float2bfloat16_rn(acc[j]);
  }
}

__global__ void __launch_bounds__(256) attend_kernel(const PrefillParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (unit >= (long long)p.T * p.heads || p.base[p.B] < 0) return;
  const int i = (int)(unit / p.heads), h = (int)(unit - (long long)i * p.heads);
  int b = 0;
  while (b + 1 < p.B && p.q_off[b + 1] <= i) ++b;
  const int q0 = p.q_off[b], q1 = p.q_off[b + 1], seq = p.seqs[b];
  const int len = seq_len(p, b);
  if (i < q0 || i >= q1 || q1 - q0 > len || seq < 0 || seq >= p.kv.max_seqs) {
    if (lane == 0) set_status(p.status, MOE_DEV_ERR_BAD_SEQ);
    return;
  }
  const int limit = len - (q1 - q0) + (i - q0) + 1;
  const int rope = p.kv.row - p.kv.rank, dim = p.dn + rope;
  float q[6], o[4];
#pragma unroll
  for (int j = 0; j < 6; ++j) q[j] = lane + 32 * j < dim ? __bfloat162float(p.q[(size_t)unit * dim + lane + 32 * j]) : 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  for (int t = 0; t < limit; ++t) {
    const size_t r = (size_t)h * p.kv_rows + p.base[b] + t;
    int page = p.kv.table[(size_t)seq * p.kv.max_blocks + (t >> p.kv.page_shift)];
    if (page < 0 || page >= p.kv.n_pages) page = 0;
    const __nv_bfloat16* kr = p.kv.pages + p.kv.row_offset(p.layer, page, t & (p.kv.page_tokens - 1)) + p.kv.rank;
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < 6; ++j) {
      const int d = lane + 32 * j;
      if (d < dim) dot = fmaf(q[j], __bfloat162float(d < p.dn ? p.k[r * p.dn + d] : kr[d - p.dn]), dot);
    }
    const float s2 = warp_sum(dot) * p.scale_log2;
    const float mn = fmaxf(m, s2);
    const float ref = mn == -INFINITY ? 0.0f : mn;
    const float f = exp2f(m - ref), w = exp2f(s2 - ref);
    l = fmaf(l, f, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = lane + 32 * j;
      if (d < p.dv) o[j] = fmaf(w, __bfloat162float(p.v[r * p.dv + d]), o[j] * f);
    }
    m = mn;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int d = lane + 32 * j;
    if (d < p.dv) p.out[(size_t)unit * p.dv + d] = __float2bfloat16_rn(o[j] / l);
  }
}

struct PrefillWs {
  size_t base, k, v, bytes;
  int rows;
};

bool prefill_shape_ok(int B, int T, int heads, int dn, int dv, int kv_tokens) {
  if ((dn != 64 && dn != 128) || (dv != 64 && dv != 128) || heads > 1024 || B > 4096) return false;
  return (long long)T * heads <= INT_MAX && ((long long)kv_tokens + 128LL * B) * heads <= INT_MAX;
}

PrefillWs prefill_ws(int B, int heads, int dn, int dv, int kv_tokens) {
  PrefillWs w;
  w.rows = (kv_tokens + kRowAlign - 1) / kRowAlign * kRowAlign + kRowAlign * (B - 1);
  w.base = 0;
  w.k = align_up((size_t)(B + 1) * sizeof(int32_t), 256);
  w.v = w.k + align_up((size_t)heads * w.rows * dn * 2, 256);
  w.bytes = w.v + align_up((size_t)heads * w.rows * dv * 2, 256);
  return w;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_latent_prefill_workspace_size(const moe_kv_cache* cache, int B, int T, int heads, int dn, int dv,
                                         int kv_tokens) {
  if (check_latent(cache, 0) != MOE_OK || B < 1 || T < 1 || heads < 1 || kv_tokens < 0) return 0;
  return prefill_shape_ok(B, T, heads, dn, dv, kv_tokens) ? prefill_ws(B, heads, dn, dv, kv_tokens).bytes : 0;
}

int moe_latent_prefill(const moe_kv_cache* cache, int layer, const void* q, const int32_t* seqs,
                       const int32_t* q_offsets, int B, int T, int heads, int dn, int dv, const void* w_kv,
                       float scale, int kv_tokens, void* out, void* ws, size_t ws_bytes, uint32_t* dev_status,
                       moe_stream_t stream) {
  int st = check_latent(cache, layer);
  if (st == MOE_ERR_INVALID_ARG || check_kv(cache) != MOE_OK) return st;
  if (B < 0 || T < 0 || heads < 1 || kv_tokens < 0 || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  const bool some = B > 0 && T > 0;
  if (some && kv_tokens < 1) return MOE_ERR_INVALID_ARG;   // a query sees its own token at least
  if (some && (!q || !seqs || !q_offsets || !w_kv || !out)) return MOE_ERR_INVALID_ARG;
  if (st != MOE_OK) return st;
  if (!prefill_shape_ok(B, T, heads, dn, dv, kv_tokens)) return MOE_ERR_UNSUPPORTED;
  if (!some) return MOE_OK;
  if (!kv_aligned(q, 16) || !kv_aligned(w_kv, 16) || !kv_aligned(out, 16)) return MOE_ERR_UNSUPPORTED;
  const PrefillWs w = prefill_ws(B, heads, dn, dv, kv_tokens);
  st = check_ws(ws, ws_bytes, w.bytes);
  if (st != MOE_OK) return st;
  char* b = reinterpret_cast<char*>(ws);
  PrefillParams p;
  p.kv = kv_view(*cache);
  p.layer = layer;
  p.B = B;
  p.T = T;
  p.heads = heads;
  p.dn = dn;
  p.dv = dv;
  p.kv_rows = w.rows;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.seqs = seqs;
  p.q_off = q_offsets;
  p.w = reinterpret_cast<const __nv_bfloat16*>(w_kv);
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.base = reinterpret_cast<int32_t*>(b + w.base);
  p.k = reinterpret_cast<__nv_bfloat16*>(b + w.k);
  p.v = reinterpret_cast<__nv_bfloat16*>(b + w.v);
  p.status = dev_status;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch_k(layout_kernel, 1, 32, 0, s, p) != cudaSuccess) return MOE_ERR_CUDA;
  if (launch_k(expand_kernel, dim3(w.rows / kTile, heads * (dn + dv) / kTile), 256, 0, s, p) != cudaSuccess)
    return MOE_ERR_CUDA;
  const long long units = (long long)T * heads;
  if (launch_k(attend_kernel, (unsigned)((units + 7) / 8), 256, 0, s, p) != cudaSuccess) return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // extern "C"
