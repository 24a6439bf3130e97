// Expanded latent attention of prompt tokens: keys and values are made per
// head from the cached latents, then a causal softmax attention reads them.
//
// plan_kernel    where each sequence's expanded rows begin, and the query blocks (calls of more than 32 sequences; else
//                expand_kernel does that)
// expand_kernel  [128 tokens] x [one head's keys and values]: latents W^T, fp32
//                sums in tensor memory, bf16 keys and f16 values into the workspace
// attend_kernel  256 query rows of one head against that head's keys and
//                values, 128 tokens at a time
//
// Values and probabilities are f16, not bf16: 11 significand bits keep their
// roundings at 2^-12 where bf16's 2^-9 on each value and probability would reach
// the output in full, at the same tensor-core rate.  The price is range: an
// expanded value beyond 65504 is clamped and reported (MOE_DEV_ERR_RANGE).
// Queries come in bf16 and keys stay bf16 beside them (one product takes one
// type): a key's rounding moves a score by about 2^-9 / sqrt(keys' width) of its
// terms' size, which the softmax averages.
//
// Measured, rank 512, rope 64, keys and values of 128:
//   5 prompts of 1..300 tokens, 32 heads     36.6 us
//   1000 tokens over 15001, 16 heads         202 us  1.12 PFLOP/s
//   8192 tokens, 32 heads                    539 us  1.40 PFLOP/s
// of which expand_kernel takes about 60 us in the last two.  4096 tokens of 16
// heads by widths (keys + rotary, values): 128 + 64, 128: 95 us (1.08 PFLOP/s); 128 +
// 0, 128: 86; 128 + 64, 64: 85; 64 + 64, 128: 84; 64, 128: 79; 64 + 64, 64: 79; 64, 64: 73
// (0.59 PFLOP/s; the forms with narrow values spill 40 to 52 bytes a thread).  70
// prompts of 64..128 tokens, 16 heads: 90 us.
#include <cfloat>
#include <cmath>

#include <cuda_fp16.h>

#include "kv_common.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kRowAlign = 128;           // sequences start at multiples of this in the expanded buffers
constexpr int kBlock = 256;              // query rows of a work item: two tiles of 128
constexpr int kTile = 128;               // tokens of a tile (and query rows of a tile)
constexpr int kChunkBytes = kTile * kBK * 2;   // 16 KB: 128 rows x 64 entries
constexpr int kThreads = 384;            // warps 0..3: producer, MMA issuer, two idle; 4..7 and 8..11: softmax
constexpr int kMaxSplits = 8;
constexpr int kTmemCols = 512;
constexpr float kGrow = 8.0f;            // log2 of the growth of a row's maximum that forces a rescaling
// Probabilities are kept as 2^7 times their ratio to the row's reference: with the growth above they reach 2^15, inside
// f16, and each is off by at most 2^-32 of the row's largest where f16's subnormals begin (unlifted 2^-25: behind one
// dominating token, a tail of many thousand small ones was lost).  Their sum carries the same factor.
constexpr float kLift = 7.0f;

struct QBlock {
  int row0, rows;   // first of its query rows in q, and how many
  int limit0;       // row r sees the tokens below limit0 + r
  int base;         // first expanded row of its sequence
};

struct TokTile {
  int seq, t0, len, pad;   // a tile of 128 expanded rows: its sequence in the cache, first token, the sequence's length
};

struct PrefillParams {
  KvView kv;
  int layer, B, T, heads, dn, dv, rope, kv_rows, max_blocks_q, sms;
  int max_splits;           // shares of a query block's tokens that there is room for
  float scale_log2;
  const __nv_bfloat16* q;
  const int32_t* seqs;
  const int32_t* q_off;
  const __nv_bfloat16* w;
  __nv_bfloat16* out;
  int32_t* counts;          // [0] query blocks, [1] next work item, [2] tiles of expanded rows, [3] shares of a block's tokens
  QBlock* blocks;
  TokTile* tiles;           // [kv_rows / 128]
  __nv_bfloat16* k;         // [heads, kv_rows, dn]
  __half* v;                // [heads, kv_rows, dv]
  __nv_bfloat16* r;         // [kv_rows, rope]
  float* part;              // with shares: [shares, heads, T, dv] unnormalised outputs
  float2* ml;               // [shares, heads, T] their (m, l)
  uint32_t* status;
};

__device__ inline int seq_len(const PrefillParams& p, int b) {
  const int s = p.seqs[b];
  return s >= 0 && s < p.kv.max_seqs ? p.kv.len_of(s) : 0;
}

// f16 of two values within its range; a NaN becomes a number as well (its token's keys are NaN and carry it to the rows
// that see the token, while a row that does not see it multiplies the value by probability 0).
__device__ inline uint32_t half2_of(float x, float y) {
  const __half2 top = __half2half2(__ushort_as_half(0x7BFFu)), h = __floats2half2_rn(x, y);   // 65504
  const __half2 c = __hmax2(__hmin2(h, top), __hneg2(top));
  return *reinterpret_cast<const uint32_t*>(&c);
}

__device__ inline uint32_t bf16x2_of(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------- plan
// One CTA.  Expanded rows: sums of the lengths rounded up to 128.  Query
// blocks: 256 rows each, a sequence's last block first (it sees most tokens, and
// long work items started first leave the shortest tail).
constexpr int kPlanThreads = 512;
constexpr int kMaxB = 4096;

__device__ inline void scan2(int (&v)[2], int (&total)[2], int (*sh)[kPlanThreads / 32]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    int inc = v[e];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) sh[e][w] = inc;
    v[e] = inc - v[e];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    int base = 0, all = 0;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
      if (i < w) base += sh[e][i];
      all += sh[e][i];
    }
    v[e] += base;
    total[e] = all;
  }
  __syncthreads();
}

// Shares of the blocks' tokens, where blocks and heads alone leave SMs idle or the longest block would run on alone.
// The estimate: a step of 128 tokens takes about 2 us, an item half a step more; items of about one length go in whole
// rounds over the SMs, others fill each other's gaps and the longest is the bound; shares cost a launch and their
// partial results, written and read at about 4 TB/s.
__device__ inline int token_shares(const PrefillParams& p, float items, float total, int longest, int shortest) {
  int best = 1;
  float least = FLT_MAX;
  for (int s = 1; s <= p.max_splits && (s == 1 || longest >= 4 * s); ++s) {
    const float rounds = ceilf(items * s / p.sms), longest_share = (float)longest / s;
    const float steps = 4 * shortest > 3 * longest ? rounds * longest_share : fmaxf(longest_share, total / p.sms);
    const float cost = 2.0f * (steps + 0.5f * rounds) + (s > 1 ? 4.0f + s * 2e-6f * p.T * p.heads * p.dv : 0.0f);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

// A sequence's part of the plan.
struct SeqPlan {
  int len, q0, n;       // tokens held; first query row and how many
  int units, blocks;    // of expanded rows (128 each), of queries
};

__device__ inline SeqPlan seq_plan(const PrefillParams& p, int b) {
  SeqPlan x = {0, 0, 0, 0, 0};
  if (b >= p.B) return x;
  const int s = p.seqs[b], q1 = p.q_off[b + 1];
  x.len = seq_len(p, b);
  x.q0 = p.q_off[b];
  const bool good = s >= 0 && s < p.kv.max_seqs && x.q0 >= 0 && q1 >= x.q0 && q1 <= p.T && q1 - x.q0 <= x.len;
  if (!good) set_status(p.status, MOE_DEV_ERR_BAD_SEQ);
  x.n = good ? q1 - x.q0 : 0;
  // in units of 128 rows, a length past the buffer as one unit too many: the sums stay small
  x.units = min((x.len + kRowAlign - 1) / kRowAlign, p.kv_rows / kRowAlign + 1);
  x.blocks = (x.n + kBlock - 1) / kBlock;
  return x;
}

// Its query blocks, the last one first; `at`: the blocks before it, `base`: its first expanded row.
__device__ inline void put_blocks(const PrefillParams& p, const SeqPlan& x, int at, int base) {
  for (int i = 0; i < x.blocks; ++i) {
    const int to = at + x.blocks - 1 - i, j0 = i * kBlock;
    if (to < p.max_blocks_q) p.blocks[to] = QBlock{x.q0 + j0, min(kBlock, x.n - j0), x.len - x.n + j0 + 1, base};
  }
}

// Tiles that a sequence's first and last block see.
__device__ inline int first_sees(const SeqPlan& x) { return (x.len - x.n + min(kBlock, x.n) + kTile - 1) / kTile; }
__device__ inline int last_sees(const SeqPlan& x) { return (x.len + kTile - 1) / kTile; }

// Up to 32 sequences need no launch for the plan: every CTA of expand_kernel finds the expanded rows for itself, and
// one warp of it writes the query blocks (plan_small).  (5 prompts of up to 300 tokens: 34.7 -> 33.0 us.)
constexpr int kSmallB = 32;

__device__ inline int warp_inclusive(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

__device__ inline void plan_small(const PrefillParams& p) {
  const int lane = threadIdx.x & 31;
  const SeqPlan x = seq_plan(p, lane);
  const int units = warp_inclusive(x.units), blocks = warp_inclusive(x.blocks);
  const long long base = (long long)(units - x.units) * kRowAlign, rows = (long long)__shfl_sync(0xffffffffu, units, 31) * kRowAlign;
  put_blocks(p, x, blocks - x.blocks, base < p.kv_rows ? (int)base : p.kv_rows);
  const int longest = __reduce_max_sync(0xffffffffu, x.blocks ? last_sees(x) : 0);
  const int shortest = __reduce_min_sync(0xffffffffu, x.blocks ? first_sees(x) : INT_MAX);
  const float total = warp_sum(x.blocks ? 0.5f * (first_sees(x) + last_sees(x)) * x.blocks : 0.0f);
  const int all = __shfl_sync(0xffffffffu, blocks, 31);
  if (lane == 0) {
    const bool fits = rows <= p.kv_rows;
    if (!fits) set_status(p.status, MOE_DEV_ERR_CAPACITY);
    p.counts[0] = fits ? min(all, p.max_blocks_q) : 0;
    p.counts[1] = 0;
    p.counts[3] = token_shares(p, (float)all * p.heads, total * p.heads, longest, shortest);
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PrefillParams p) {
  __shared__ int sh[2][kPlanThreads / 32];
  __shared__ int s_base[kMaxB], s_len[kMaxB];   // first expanded row and length of each sequence
  __shared__ int s_longest, s_shortest;         // tiles of tokens that a block of queries sees
  __shared__ unsigned long long s_total;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    s_longest = 0;
    s_shortest = INT_MAX;
    s_total = 0;
  }
  __syncthreads();
  long long rows = 0;
  int blocks = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    const SeqPlan x = seq_plan(p, b);
    int v[2] = {x.units, x.blocks}, total[2];
    scan2(v, total, sh);
    if (b < p.B) {
      const long long at = rows + (long long)v[0] * kRowAlign;
      const int base = at < p.kv_rows ? (int)at : p.kv_rows;
      s_base[b] = base;
      s_len[b] = x.len;
      if (p.max_splits > 1 && x.blocks > 0) {
        atomicMin(&s_shortest, first_sees(x));
        atomicMax(&s_longest, last_sees(x));
        atomicAdd(&s_total, (unsigned long long)(first_sees(x) + last_sees(x)) * x.blocks);    // twice the sum, as if in even steps
      }
      put_blocks(p, x, blocks + v[1], base);
    }
    rows += (long long)total[0] * kRowAlign;
    blocks += total[1];
  }
  const bool fits = rows <= p.kv_rows;
  __syncthreads();
  if (threadIdx.x == 0) {
    if (!fits) set_status(p.status, MOE_DEV_ERR_CAPACITY);
    p.counts[3] = token_shares(p, (float)blocks * p.heads, 0.5f * (float)s_total * p.heads, s_longest, s_shortest);
    p.counts[0] = fits ? min(blocks, p.max_blocks_q) : 0;
    p.counts[1] = 0;
    p.counts[2] = fits ? (int)(rows / kRowAlign) : 0;
  }
  if (!fits) return;
  __syncthreads();
  for (int t = threadIdx.x; t < (int)(rows / kRowAlign); t += kPlanThreads) {
    const int row = t * kRowAlign;
    int lo = 0, hi = p.B;   // the last b with base <= row; sequences without tokens own no row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_base[mid] <= row) lo = mid;
      else hi = mid;
    }
    p.tiles[t] = TokTile{p.seqs[lo], row - s_base[lo], s_len[lo], 0};
  }
}

// ---------------------------------------------------------------- expand
// D[128 tokens, one head's dn + dv features] = latents W_head^T, rank deep: the
// latents of a token tile stay in shared memory (rank x 128 x 2 bytes) while the
// CTA's heads' weights pass by in 64-deep stages, so a unit reads only its
// weights.  Two accumulators in tensor memory (columns 0 and 256): the epilogue
// of one unit runs under the products of the next.  Rows past a sequence's end
// are written as zeros (the attention multiplies them by probability 0).
// 16000 tokens of 16 heads: 60 us for 67 GFLOP and 134 MB of keys and values, about 4200 cycles of products in the 6000
// that a unit takes; without the stores it would take 4900, so it is the way of the 134 MB through L2 that bounds it.
// Weights split over a pair of CTAs (half the reads of them), stores by TMA from shared memory and both L2 policies
// made no difference.
// Warp 0 = TMA, warp 1 = MMA (and TMEM owner), warps 2..9 = epilogue (4 lane
// quarters x 2 halves of the features: with 4 warps the epilogue took 7200
// cycles a unit against 4100 of products), warps 10, 11 = rotary keys.
constexpr int kExThreads = 384;
constexpr int kExStages = 3;
constexpr int kExStage = 256 * kBK * 2;    // 32 KB of weights
constexpr int kMaxChunks = 512 / kBK;

struct ExShared {
  uint64_t a_full[kMaxChunks], a_empty, b_full[kExStages], b_empty[kExStages], d_full[2], d_empty[2], drain;
  uint32_t tmem;
  int abort;
  int tiles, base[kSmallB], len[kSmallB], ids[kSmallB];   // up to 32 sequences: tiles, and each one's first tile, length, id
};

// A tile of 128 expanded rows: its sequence, first token and the sequence's length.
__device__ inline int4 tile_of(const PrefillParams& p, const ExShared& sh, int tile) {
  if (p.B > kSmallB) return __ldg(reinterpret_cast<const int4*>(p.tiles + tile));
  int b = 0;
  for (int i = 1; i < p.B; ++i)
    if (sh.base[i] <= tile) b = i;            // the last one that begins at or before it: those without tokens own none
  return make_int4(sh.ids[b], (tile - sh.base[b]) * kTile, sh.len[b], 0);
}

// 32 bytes at once: a whole sector of one row per thread.
__device__ inline void st_sector(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__global__ void __launch_bounds__(kExThreads, 1)
expand_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
              const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ExShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunks = p.kv.rank / kBK, N = p.dn + p.dv;
  if (tid == 0) {
    for (int c = 0; c < chunks; ++c) mbar_init(&sh.a_full[c], 1);
    mbar_init(&sh.a_empty, 1);
    for (int i = 0; i < kExStages; ++i) {
      mbar_init(&sh.b_full[i], 1);
      mbar_init(&sh.b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.d_full[i], 1);
      mbar_init(&sh.d_empty[i], 8);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 64) {
    prefetch_map(&map_x);
    prefetch_map(&map_w);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();
  if (p.B <= kSmallB && warp == 2) {
    const int len = lane < p.B ? seq_len(p, lane) : 0;
    const int n = min((len + kRowAlign - 1) / kRowAlign, p.kv_rows / kRowAlign + 1), sum = warp_inclusive(n);
    sh.base[lane] = sum - n;
    sh.len[lane] = len;
    sh.ids[lane] = lane < p.B ? p.seqs[lane] : 0;
    if (lane == 31) sh.tiles = (long long)sum * kRowAlign <= p.kv_rows ? sum : 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_flag = &sh.abort;
  const int tiles = p.B <= kSmallB ? sh.tiles : p.counts[2];
  const int total = tiles * p.heads;                       // units: token tile major, head minor
  const int per = (total + gridDim.x - 1) / gridDim.x;
  const int u0 = min(total, (int)blockIdx.x * per), u1 = min(total, u0 + per);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    const uint32_t smem0 = uni(smem_u32(smem)), b0 = smem0 + chunks * kChunkBytes;
    const uint32_t af = uni(smem_u32(&sh.a_full[0])), bf = uni(smem_u32(&sh.b_full[0]));
    const int page = p.kv.page_tokens, box = page;
    int loaded = 0, stage = 0, fills = 0;
    uint32_t par = 1;
    bool ok = true;
    auto load_w = [&](int head, int c) {
      ok = ok && warp_wait(&sh.b_empty[stage], par, abort_flag);
      if (!ok) return;
      mbar_expect_tx_warp(bf + 8 * stage, (uint32_t)(N * 128));
      tma_load_2d_warp(b0 + stage * kExStage, &map_w, bf + 8 * stage, c * kBK, head * N);
      ++fills;
      if (++stage == kExStages) {
        stage = 0;
        par ^= 1u;
      }
    };
    for (int u = u0; ok && u < u1; ++u) {
      const int tile = u / p.heads, head = u - tile * p.heads;
      int c0 = 0;
      if (u == u0 || head == 0) {                          // another token tile
        const int4 d = tile_of(p, sh, tile);   // sequence, first token, length
        const int nb = (int)uni((min(kTile, d.z - d.y) + box - 1) / box);
        int row = 0;
        if (lane < nb) {
          int pg = p.kv.table[(size_t)d.x * p.kv.max_blocks + ((d.y + lane * box) >> p.kv.page_shift)];
          if (pg < 0 || pg >= p.kv.n_pages) {
            set_status(p.status, MOE_DEV_ERR_BAD_PAGE);
            pg = 0;
          }
          row = (p.layer * p.kv.n_pages + pg) * page;
        }
        int rows[kTile / 16];
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i) rows[i] = (int)uni(lane == i ? row : 0);
        ok = warp_wait(&sh.a_empty, (loaded & 1) ^ 1u, abort_flag);
        if (!ok) break;
        ++loaded;
        for (int c = 0; c < chunks; ++c) {
          mbar_expect_tx_warp(af + 8 * c, (uint32_t)(nb * box * 128));
#pragma unroll
          for (int i = 0; i < kTile / 16; ++i)
            if (i < nb) tma_load_2d_warp(smem0 + c * kChunkBytes + i * box * 128, &map_x, af + 8 * c, c * kBK, rows[i]);
          if (c < kExStages) load_w(head, c);              // between them: the first product needs both
        }
        if (!ok) break;
        c0 = min(chunks, kExStages);
      }
      for (int c = c0; ok && c < chunks; ++c) load_w(head, c);
    }
    volatile int no_abort = 0;
    if (loaded)
      for (int c = 0; c < chunks; ++c) mbar_wait(&sh.a_full[c], (loaded - 1) & 1, &no_abort);
    for (int i = 0; i < kExStages; ++i) {
      const int n = fills / kExStages + (fills % kExStages > i ? 1 : 0);
      if (n > 0) mbar_wait(&sh.b_full[i], (n - 1) & 1, &no_abort);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    const uint32_t tm = uni(tmem), smem0 = uni(smem_u32(smem));
    const uint64_t da0 = smem_desc(smem0), db0 = smem_desc(smem0 + chunks * kChunkBytes);
    const uint32_t idesc = make_idesc(128, N);
    int loaded = 0, stage = 0, n = 0;
    uint32_t par = 0;
    bool ok = true, issued = false;
    for (int u = u0; ok && u < u1; ++u, ++n) {
      const int head = u % p.heads, buf = n & 1;
      if (u == u0 || head == 0) ++loaded;
      ok = warp_wait(&sh.d_empty[buf], ((n >> 1) & 1) ^ 1u, abort_flag);
      for (int c = 0; ok && c < chunks; ++c) {
        ok = warp_wait(&sh.a_full[c], (loaded - 1) & 1, abort_flag) && warp_wait(&sh.b_full[stage], par, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint64_t da = da0 + ((uint64_t)(c * kChunkBytes) >> 4), db = db0 + ((uint64_t)(stage * kExStage) >> 4);
#pragma unroll
        for (int k = 0; k < kBK / kUK; ++k)
          tc_mma_warp(tm + buf * 256, da + ((k * kUK * 2) >> 4), db + ((k * kUK * 2) >> 4), idesc, k ? 1u : (c ? 1u : 0u));
        issued = true;
        tc_commit_warp(&sh.b_empty[stage]);
        if (++stage == kExStages) {
          stage = 0;
          par ^= 1u;
        }
      }
      if (!ok) break;
      tc_commit_warp(&sh.d_full[buf]);
      if (head == p.heads - 1) tc_commit_warp(&sh.a_empty);
    }
    if (issued) {
      volatile int no_abort = 0;
      tc_commit_warp(&sh.drain);
      mbar_wait(&sh.drain, 0, &no_abort);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ------------------------------------------------ rotary keys, once per token: 16 bytes a thread, neighbours in a row
    const int vecs = p.rope / 8;
    if (p.B <= kSmallB && warp == 11 && blockIdx.x == gridDim.x - 1) plan_small(p);   // the CTA with the least to do
    for (int u = u0; u < u1; ++u) {
      const int tile = u / p.heads;
      if (u != tile * p.heads) continue;                   // the CTA that has the tile's first head
      const int4 d = tile_of(p, sh, tile);
#pragma unroll 4
      for (int x = tid - 320; x < kTile * vecs; x += 64) {
        const int r = x / vecs, y = x - r * vecs, t = d.y + r;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (t < d.z) {
          int pg = p.kv.table[(size_t)d.x * p.kv.max_blocks + (t >> p.kv.page_shift)];
          if (pg < 0 || pg >= p.kv.n_pages) pg = 0;
          v = __ldg(reinterpret_cast<const uint4*>(p.kv.pages + p.kv.row_offset(p.layer, pg, t & (p.kv.page_tokens - 1)) +
                                                   p.kv.rank) + y);
        }
        reinterpret_cast<uint4*>(p.r + ((size_t)tile * kTile + r) * p.rope)[y] = v;
      }
    }
  } else {
    // ------------------------------------------------ epilogue: a thread owns a token row and half the features
    const int quarter = warp & 3, half = (warp - 2) >> 2, r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const int c0 = half ? N / 64 * 32 : 0, c1 = half ? N : N / 64 * 32;      // its features, in blocks of 32
    int n = 0;
    uint32_t mask = 0;
    bool clamped = false;
    for (int u = u0; u < u1; ++u, ++n) {
      const int tile = u / p.heads, head = u - tile * p.heads, buf = n & 1;
      if (u == u0 || head == 0) {
        const int4 d = tile_of(p, sh, tile);
        mask = d.y + r < d.z ? 0xFFFFFFFFu : 0u;                             // rows past the end: zeros
      }
      if (!warp_wait(&sh.d_full[buf], (n >> 1) & 1, abort_flag)) break;
      tc_fence_after();
      const size_t at = (size_t)head * p.kv_rows + tile * kTile + r;
      uint32_t v[2][32];
      const uint32_t col = lane_base + buf * 256;
      tmem_ld32(col + c0, v[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 32 * i;
        if (c >= c1) break;
        tmem_ld_wait();
        if (c + 32 < c1) tmem_ld32(col + c + 32, v[(i + 1) & 1]);
        const uint32_t(&x)[32] = v[i & 1];
        uint32_t o[16];
        void* dst;
        if (c < p.dn) {
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            // k + 0 k: an infinite key becomes NaN.  Its token's values are infinite too, clamped below, and the score it
            // would give may be -infinity: probability 0 times a finite value would hide it.
            const float2 k = make_float2(__uint_as_float(x[2 * y]), __uint_as_float(x[2 * y + 1]));
            const float2 z = fma2(k, make_float2(0.0f, 0.0f), k);
            o[y] = bf16x2_of(z.x, z.y) & mask;
          }
          dst = p.k + at * p.dn + c;
        } else {
          float big = 0.0f;
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const float e0 = __uint_as_float(x[2 * y]), e1 = __uint_as_float(x[2 * y + 1]);
            big = fmaxf(big, fmaxf(fabsf(e0), fabsf(e1)));
            o[y] = half2_of(e0, e1) & mask;
          }
          clamped |= (big > 65504.0f) & (mask != 0u);
          dst = p.v + at * p.dv + c - p.dn;
        }
        st_sector(dst, o);
        st_sector((char*)dst + 32, o + 8);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.d_empty[buf]);
    }
    if (clamped) set_status(p.status, MOE_DEV_ERR_RANGE);
  }
  __syncthreads();
  if (*abort_flag && tid == 0) set_status(p.status, MOE_DEV_ERR_TIMEOUT);
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// ---------------------------------------------------------------- attention
// S = Q K^T and O = P V for two tiles of 128 query rows in turn, 128 tokens a step, flash-style: running maximum and sum
// per row in fp32, O rescaled only when the maximum rises by more than 2^8.  P replaces its S in tensor memory and is the
// value product's A operand from there, so only V is read from shared memory.
// Bound: 2600 cycles of products a step and 2625 of shared memory (S alone reads 126 bytes a cycle); a step takes 3400
// to 3600, the rest lies between groups of products (their queue covers about 90 cycles, a look at a barrier takes 80)
// and in the wait for K(i+1), whose place in the ring comes free 1500 cycles before its use.  8192 tokens, 32 heads:
// 687 GFLOP in about 465 us, 76% of the measured bf16 peak.
//
// Product with the A operand in tensor memory (16-bit entries, two to a column), one elected lane of a warp issuing.
__device__ inline void tc_mma_ta_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accum)
      : "memory");
}

// Which of three barriers are past their phases (bits 0, 1, 2); does not wait.
__device__ inline uint32_t test_three(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint64_t* c, uint32_t pc) {
  uint32_t x, y, z;
  asm volatile(
      "{\n .reg .pred p, q, r;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%3], %4;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 q, [%5], %6;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 r, [%7], %8;\n"
      " selp.u32 %0, 1, 0, p;\n selp.u32 %1, 2, 0, q;\n selp.u32 %2, 4, 0, r;\n}\n"
      : "=r"(x), "=r"(y), "=r"(z)
      : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb), "r"(smem_u32(c)), "r"(pc)
      : "memory");
  return x | y | z;
}

// fp32 accumulation, f16 operands, A and B K-major
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }
struct Shared {
  uint64_t full[4], empty[4];                    // key (with their rotary part) and value tiles
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_ready[2], o_full[2];
  uint64_t w_full[2], w_empty[2];                // work items
  uint64_t drain;
  int item[2];
  uint32_t tmem;
  int abort;
};

// Shared memory by the chunks of 64 entries of a query (KC: with the rotary part): two query tiles, two rotary key
// tiles, and a ring of key and value tiles in the order of their use, K(0) V(0) K(1) V(1) ...: while V(i) and K(i+1)
// are read, V(i+1) is on its way.
template <int KC>
struct Attend {
  static constexpr int kQ = KC * kChunkBytes, kUnit = 2 * kChunkBytes;
  static constexpr int kUnits = KC == 3 ? 3 : 4;
  static constexpr int kRope = 2 * kQ, kRing = kRope + 2 * kChunkBytes;   // where the parts begin
  static constexpr int kSmem = kRing + kUnits * kUnit + 1024;
};

// A work item: 256 query rows of one head against one of `splits` shares of their tokens.
struct Item {
  int head, row0, rows, limit0, base, block, split;
  int first, tiles[2];   // its first tile of tokens, and how many each query tile takes
};

__device__ inline bool get_item(const PrefillParams& p, int k, int n_blocks, int splits, int group, Item& it) {
  if (k >= n_blocks * p.heads * splits) return false;
  // heads in groups that fill the grid once, so that a group's keys and values are read while they are in L2
  const int units = n_blocks * splits, per = units * group, gi = k / per, in = k - gi * per;
  const int gh = min(group, p.heads - gi * group), x = in / gh;
  it.head = gi * group + (in - x * gh);
  it.block = x / splits;
  it.split = x - it.block * splits;
  const int4 qb = __ldg(reinterpret_cast<const int4*>(p.blocks + it.block));
  it.row0 = qb.x;
  it.rows = qb.y;
  it.limit0 = qb.z;
  it.base = qb.w;
  const int all = (it.limit0 + it.rows - 1 + kTile - 1) / kTile;   // the last row sees the most
  const int from = (int)((long long)all * it.split / splits), to = (int)((long long)all * (it.split + 1) / splits);
  it.first = from;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int last = min(it.rows, (g + 1) * kTile) - 1;
    const int mine = last >= g * kTile ? (it.limit0 + last + kTile - 1) / kTile : 0;
    it.tiles[g] = max(0, min(mine, to) - from);
  }
  return true;
}

template <int KC, int VC>
__global__ void __launch_bounds__(kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_v,
              const PrefillParams p) {
  using A = Attend<KC>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < A::kUnits; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sh.q_full[g], 1);
      mbar_init(&sh.q_empty[g], 1);
      mbar_init(&sh.s_full[g], 1);
      mbar_init(&sh.p_ready[g], 4);
      mbar_init(&sh.o_full[g], 1);
      mbar_init(&sh.w_full[g], 1);
      mbar_init(&sh.w_empty[g], 9);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 64) {
    prefetch_map(&map_q);
    prefetch_map(&map_k);
    prefetch_map(&map_r);
    prefetch_map(&map_v);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_flag = &sh.abort;
  const int n_blocks = p.counts[0], splits = p.counts[3];
  const int group = n_blocks ? max(1, min(p.heads, (int)gridDim.x / (n_blocks * splits))) : 1;
  const int rope_chunk = p.rope ? 1 : 0, key_chunks = KC - rope_chunk;
  Item it;
  // A softmax thread holds a row of 128 scores: the first four warps give registers to the other eight
  // (128 threads x (104 + 200 + 200) = 384 x 168, what the launch has).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0) {
      // ---------------------------------------------- work items and TMA
      const uint32_t smem0 = uni(smem_u32(smem));
      const uint32_t full0 = uni(smem_u32(&sh.full[0]));
      const uint32_t qf = uni(smem_u32(&sh.q_full[0]));
      int n = 0, units = 0, slot = 0, ropes = 0, q_loads0 = 0, q_loads1 = 0;
      uint32_t par = 1;
      bool ok = true;
      // `chunks` of 64 columns of 128 rows into the next place of the ring.  A key tile's rotary part goes into the
      // buffer its last-but-one predecessor had, which is over before the ring's place is free.
      auto load_unit = [&](const CUtensorMap* map, int chunks, int row, bool rope, int rope_row) {
        if (!ok) return;
        ok = warp_wait(&sh.empty[slot], par, abort_flag);
        if (!ok) return;
        ++units;
        mbar_expect_tx_warp(full0 + 8 * slot, (uint32_t)((chunks + (rope ? 1 : 0)) * kChunkBytes));
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (c < chunks)
            tma_load_2d_warp(smem0 + A::kRing + slot * A::kUnit + c * kChunkBytes, map, full0 + 8 * slot, c * kBK, row);
        if (rope)
          tma_load_2d_warp(smem0 + A::kRope + (ropes++ & 1) * kChunkBytes, &map_r, full0 + 8 * slot, 0, rope_row);
        if (++slot == A::kUnits) {
          slot = 0;
          par ^= 1u;
        }
      };
      auto load_k = [&](int head, int row) { load_unit(&map_k, key_chunks, head * p.kv_rows + row, rope_chunk != 0, row); };
      auto load_q = [&](int g, int& loads, int head, int row0) {
        ok = warp_wait(&sh.q_empty[g], (loads & 1) ^ 1u, abort_flag);
        if (!ok) return;
        ++loads;
        mbar_expect_tx_warp(qf + 8 * g, A::kQ);
#pragma unroll
        for (int c = 0; c < KC; ++c)
          tma_load_2d_warp(smem0 + g * A::kQ + c * kChunkBytes, &map_q, qf + 8 * g, head * (p.dn + p.rope) + c * kBK,
                           row0 + g * kTile);
      };
      // The next work item's number, for everyone.  Fetched before the current item's last tile is asked for: early enough
      // to hide the atomic, late enough that the items go to whoever is free (a whole item earlier, 8192 tokens of 8
      // heads took 237 us instead of 155).
      auto fetch = [&]() {
        int k = 0;
        ok = warp_wait(&sh.w_empty[n & 1], ((n >> 1) & 1) ^ 1u, abort_flag);
        if (!ok) return 0;
        if (lane == 0) {
          k = atomicAdd(&p.counts[1], 1);
          sh.item[n & 1] = k;
          mbar_arrive(&sh.w_full[n & 1]);
        }
        ++n;
        return (int)uni(k);
      };
      int ahead = fetch();
      while (ok) {
        if (!__any_sync(0xffffffffu, get_item(p, ahead, n_blocks, splits, group, it))) break;
        const int row0 = (int)uni(it.row0), head = (int)uni(it.head), base = (int)uni(it.base + it.first * kTile);
        const int ta = (int)uni(it.tiles[0]), tb = (int)uni(it.tiles[1]), tiles = max(ta, tb);
        if (ta) load_q(0, q_loads0, head, row0);
        if (ok && tiles) load_k(head, base);
        if (ok && tb) load_q(1, q_loads1, head, row0);
        if (!tiles) ahead = fetch();
        for (int i = 0; i < tiles && ok; ++i) {
          if (i + 1 == tiles) ahead = fetch();
          if (ok) load_unit(&map_v, VC, head * p.kv_rows + base + i * kTile, false, 0);
          if (ok && i + 1 < tiles) load_k(head, base + (i + 1) * kTile);
        }
        if (!ok) break;
      }
      // drain: whatever was asked for lands before the CTA can exit
      volatile int no_abort = 0;
      if (q_loads0) mbar_wait(&sh.q_full[0], (q_loads0 - 1) & 1, &no_abort);
      if (q_loads1) mbar_wait(&sh.q_full[1], (q_loads1 - 1) & 1, &no_abort);
      for (int i = 0; i < A::kUnits; ++i) {
        const int loads = units / A::kUnits + (units % A::kUnits > i ? 1 : 0);
        if (loads > 0) mbar_wait(&sh.full[i], (loads - 1) & 1, &no_abort);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------- MMA issuer
      // Order for tiles a, b: S_a(0) S_b(0) | PV_a(i) S_a(i+1) PV_b(i) S_b(i+1): while one tile's softmax runs, the
      // other tile's products do.  P lies in its S's columns, so S_a(i+1) follows PV_a(i).
      const uint32_t tm = uni(tmem), smem0 = uni(smem_u32(smem));
      const uint64_t dq0 = smem_desc(smem0), dk0 = smem_desc(smem0 + A::kRing), dr0 = smem_desc(smem0 + A::kRope);
      const uint64_t dv0 = smem_desc_mn(smem0 + A::kRing, kChunkBytes);
      constexpr uint32_t idesc_s = make_idesc(128, kTile), idesc_v = idesc_f16(128, VC * kBK) | kTransB;
      constexpr int KN = KC < 2 ? KC : 2;      // key chunks at most
      const int rope_steps = (int)uni(p.rope / kUK);
      int n = 0, ropes = 0, q_uses0 = 0, q_uses1 = 0, p_uses0 = 0, p_uses1 = 0;
      int slot = 0;                            // the ring's next tile
      uint32_t par = 0;
      bool issued = false, ok = true;
      auto step = [&](int& at, uint32_t& parity) {
        if (++at == A::kUnits) {
          at = 0;
          parity ^= 1u;
        }
      };
      auto issue_s = [&](int g, int at) {
        const uint64_t dq = dq0 + (uint64_t)((g * A::kQ) >> 4), dk = dk0 + (uint64_t)((at * A::kUnit) >> 4);
        const uint64_t dr = dr0 + (uint64_t)(((ropes & 1) * kChunkBytes) >> 4);
#pragma unroll
        for (int c = 0; c < KN; ++c)
          if (c < key_chunks)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              tc_mma_warp(tm + g * kTile, dq + ((c * kChunkBytes + x * kUK * 2) >> 4),
                          dk + ((c * kChunkBytes + x * kUK * 2) >> 4), idesc_s, (c | x) ? 1u : 0u);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x < rope_steps)
            tc_mma_warp(tm + g * kTile, dq + (((KC - 1) * kChunkBytes + x * kUK * 2) >> 4), dr + ((x * kUK * 2) >> 4),
                        idesc_s, 1u);
        tc_commit_warp(&sh.s_full[g]);
        issued = true;
      };
      auto issue_pv = [&](int g, int at, uint32_t acc) {
        const uint64_t dv = dv0 + (uint64_t)((at * A::kUnit) >> 4);
#pragma unroll
        for (int x = 0; x < kTile / kUK; ++x)
          tc_mma_ta_warp(tm + 256 + g * kTile, tm + g * kTile + x * 8, dv + ((x * kUK * 128) >> 4), idesc_v, x ? 1u : acc);
      };
      for (;;) {
        ok = warp_wait(&sh.w_full[n & 1], (n >> 1) & 1, abort_flag);
        if (!ok) break;
        const int k = (int)uni(sh.item[n & 1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.w_empty[n & 1]);
        ++n;
        if (!__any_sync(0xffffffffu, get_item(p, k, n_blocks, splits, group, it))) break;
        const int ta = (int)uni(it.tiles[0]), tb = (int)uni(it.tiles[1]), tiles = max(ta, tb);
        if (!tiles) continue;
        ok = warp_wait(&sh.full[slot], par, abort_flag);
        if (!ok) break;
        if (ta) {
          ok = warp_wait(&sh.q_full[0], q_uses0 & 1, abort_flag);
          if (!ok) break;
          ++q_uses0;
          tc_fence_after();
          issue_s(0, slot);
          if (ta == 1) tc_commit_warp(&sh.q_empty[0]);
        }
        if (tb) {
          ok = warp_wait(&sh.q_full[1], q_uses1 & 1, abort_flag);
          if (!ok) break;
          ++q_uses1;
          tc_fence_after();
          issue_s(1, slot);
          if (tb == 1) tc_commit_warp(&sh.q_empty[1]);
        }
        step(slot, par);
        ++ropes;
        // The products' queue is short (a few instructions), so whatever stands between two groups of them shows: one
        // look at the barriers of tile a's two products, and few commits (the softmax warps let go of the keys' places;
        // the values' go back here, at once).  Tile b sees at least what a sees.
        for (int i = 0; i < tiles; ++i) {
          const uint32_t acc = i ? 1u : 0u;
          const bool more = i + 1 < tiles, in_a = i < ta;
          int sk = slot;                                       // K(i+1); slot is V(i)'s
          uint32_t pk = par;
          step(sk, pk);
          uint64_t* const p_bar = in_a ? &sh.p_ready[0] : &sh.full[slot];
          const uint32_t p_par = in_a ? p_uses0 & 1 : par;
          const uint32_t seen = __reduce_and_sync(
              0xffffffffu, test_three(&sh.full[slot], par, p_bar, p_par, &sh.full[more ? sk : slot], more ? pk : par));
          ok = ((seen & 1) || warp_wait(&sh.full[slot], par, abort_flag)) && ((seen & 2) || warp_wait(p_bar, p_par, abort_flag));
          if (!ok) break;
          tc_fence_after();
          if (in_a) {
            ++p_uses0;
            issue_pv(0, slot, acc);
            if (i + 1 == ta) tc_commit_warp(&sh.o_full[0]);
            if (!tb) tc_commit_warp(&sh.empty[slot]);
          }
          if (more && !(seen & 4)) {
            ok = warp_wait(&sh.full[sk], pk, abort_flag);
            if (!ok) break;
            tc_fence_after();
          }
          if (i + 1 < ta) {
            issue_s(0, sk);
            if (i + 2 == ta) tc_commit_warp(&sh.q_empty[0]);
          }
          if (i < tb) {
            ok = warp_wait(&sh.p_ready[1], p_uses1++ & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            issue_pv(1, slot, acc);
            if (i + 1 == tb) tc_commit_warp(&sh.o_full[1]);
            tc_commit_warp(&sh.empty[slot]);
          }
          if (i + 1 < tb) {
            issue_s(1, sk);
            if (i + 2 == tb) tc_commit_warp(&sh.q_empty[1]);
          }
          slot = sk;
          par = pk;
          if (more) {
            step(slot, par);                                   // V(i+1); else the next item's K(0)
            ++ropes;
          }
        }
        if (!ok) break;
      }
      if (issued) {   // every issued product completes before tensor memory is released
        volatile int no_abort = 0;
        tc_commit_warp(&sh.drain);
        mbar_wait(&sh.drain, 0, &no_abort);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ------------------------------------------------ softmax: tile g = 0 in warps 4..7, 1 in warps 8..11; a thread owns a row
    const int g = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_col = lane_base + g * kTile, o_col = lane_base + 256 + g * kTile;
    int n = 0, uses = 0, steps = 0;
    bool ok = true;
    const float scale = p.scale_log2;
    const bool neg = scale < 0.0f;
    const float unseen = neg ? INFINITY : -INFINITY;   // what a token out of sight scores
    // A key tile's last reader is tile b's S (a's, without a b): when it is known to be over, one lane of that tile's warps
    // lets go of the place.
    int at_k = 0;   // the place of the step's keys
    // the next work item with tokens for this tile
    auto next_item = [&]() {
      for (;;) {
        ok = warp_wait(&sh.w_full[n & 1], (n >> 1) & 1, abort_flag);
        if (!ok) return false;
        const int k = sh.item[n & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.w_empty[n & 1]);
        ++n;
        if (!__any_sync(0xffffffffu, get_item(p, k, n_blocks, splits, group, it))) return false;
        if (g ? it.tiles[1] : it.tiles[0]) return true;
        at_k = (at_k + 2 * max(it.tiles[0], it.tiles[1])) % A::kUnits;
      }
    };
    bool have = next_item();
    while (have) {
      const int tiles = g ? it.tiles[1] : it.tiles[0], first = it.first, in_block = g * kTile + r;
      const int limit = it.limit0 + in_block - first * kTile;
      const bool mine = in_block < it.rows, releases = g == 1 || it.tiles[1] == 0;
      float m = -INFINITY, l = 0.0f;
      for (int i = 0; i < tiles; ++i, ++steps) {
        ok = warp_wait(&sh.s_full[g], steps & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (releases && quarter == 0 && lane == 0) mbar_arrive(&sh.empty[at_k]);
        at_k = at_k + 2 >= A::kUnits ? at_k + 2 - A::kUnits : at_k + 2;
        float s[kTile];
        uint32_t(&u)[kTile] = reinterpret_cast<uint32_t(&)[kTile]>(s);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&u[32 * c]));
        tmem_ld_wait();
        const int see = limit - i * kTile;
        if (!__all_sync(0xffffffffu, see >= kTile)) {   // on the diagonal and past the end: out of sight
#pragma unroll
          for (int j = 0; j < kTile; ++j)
            if (j >= see) s[j] = unseen;
        }
        float t4[4] = {s[0], s[1], s[2], s[3]};
        if (!neg) {
#pragma unroll
          for (int j = 4; j < kTile; j += 8)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              t4[x] = j + 4 + x < kTile ? fmaxf(t4[x], fmaxf(s[j + x], s[j + 4 + x])) : fmaxf(t4[x], s[j + x]);
        } else {
#pragma unroll
          for (int j = 4; j < kTile; ++j) t4[j & 3] = fminf(t4[j & 3], s[j]);
        }
        float top = neg ? fminf(fminf(t4[0], t4[1]), fminf(t4[2], t4[3])) : fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        top = see > 0 ? top * scale : -INFINITY;
        bool grow = false;
        float f = 1.0f;
        if (top > m) {
          if (m == -INFINITY) {
            m = top;
          } else if (top > m + kGrow) {
            f = ex2(m - top);
            l *= f;
            m = top;
            grow = true;
          }
        }
        if (__any_sync(0xffffffffu, grow)) {
          // this S was issued behind the previous value product, so O is complete; the lanes are this warp's alone
          for (int c = 0; c < VC * kBK; c += 16) {
            uint32_t v[16];
            tmem_ld16(o_col + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * f);
            tmem_st16(o_col + c, v);
          }
        }
        const float ref = m == -INFINITY ? 0.0f : m - kLift;
        float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 x = fma2(make_float2(s[32 * c + 2 * j], s[32 * c + 2 * j + 1]), make_float2(scale, scale),
                            make_float2(-ref, -ref));
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            if (j & 1) sum1 = add2(sum1, x);
            else sum0 = add2(sum0, x);
            const __half2 h = __floats2half2_rn(x.x, x.y);
            pk[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          tmem_st16(s_col + 16 * c, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[g]);
        l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
      }
      if (!ok) break;
      if (!g) at_k = (at_k + 2 * (max(it.tiles[0], it.tiles[1]) - tiles)) % A::kUnits;   // a's item goes on without it
      // where this item's results go; the next item's numbers come before the wait for the last product
      const size_t row = (size_t)it.row0 + in_block;
      const int head = it.head, split = it.split;
      have = next_item();
      if (!have && !ok) break;
      if (!warp_wait(&sh.o_full[g], uses++ & 1, abort_flag)) break;
      tc_fence_after();
      const bool parts = splits > 1;
      const size_t at = parts ? ((size_t)split * p.heads + head) * p.T + row : row * p.heads + head;
      if (parts && mine) p.ml[at] = make_float2(m, l);
      const float inv_l = 1.0f / l;
      uint32_t v[2][32];
      tmem_ld32(o_col, v[0]);
#pragma unroll
      for (int c = 0; c < VC * kBK; c += 32) {
        uint32_t(&x)[32] = v[(c >> 5) & 1];
        tmem_ld_wait();
        if (c + 32 < VC * kBK) tmem_ld32(o_col + c + 32, v[((c >> 5) + 1) & 1]);
        if (parts) {
          if (mine) {
#pragma unroll
            for (int y = 0; y < 4; ++y) st_sector(p.part + at * (VC * kBK) + c + 8 * y, x + 8 * y);
          }
        } else {
          uint32_t w[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) w[y] = bf16x2_of(__uint_as_float(x[2 * y]) * inv_l, __uint_as_float(x[2 * y + 1]) * inv_l);
          if (mine) {
            st_sector(p.out + at * (VC * kBK) + c, w);
            st_sector(p.out + at * (VC * kBK) + c + 16, w + 8);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (*abort_flag && tid == 0) set_status(p.status, MOE_DEV_ERR_TIMEOUT);
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// ---------------------------------------------------------------- combine of the token shares
// The shares' outputs weighted by their (m, l), in share order: a thread has four entries of a (query row, head), and
// its shares' values are asked for together with their statistics.  A share in which the row's tile had no tokens wrote
// nothing: which ones did follows from the block, as in get_item.
__global__ void __launch_bounds__(256) combine_splits_kernel(const PrefillParams p) {
  pdl_wait();
  pdl_trigger();
  const int block = blockIdx.x, splits = p.counts[3];
  if (block >= p.counts[0] || splits == 1) return;
  const int4 qb = __ldg(reinterpret_cast<const int4*>(p.blocks + block));
  const int all = (qb.z + qb.y - 1 + kTile - 1) / kTile, vecs = p.dv / 4;
  for (int x = blockIdx.y * blockDim.x + threadIdx.x; x < qb.y * p.heads * vecs; x += gridDim.y * blockDim.x) {
    const int v = x % vecs, y = x / vecs, j = y / p.heads, head = y - j * p.heads;
    const int last = min(qb.y, (j / kTile + 1) * kTile) - 1, mine = (qb.z + last + kTile - 1) / kTile;
    const size_t row = (size_t)qb.x + j;
    float2 ml[kMaxSplits];
    float4 o[kMaxSplits];
    float ref = -INFINITY;
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s) {
      ml[s] = make_float2(-INFINITY, 0.0f);
      o[s] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (s < splits && (int)((long long)all * s / splits) < min(mine, (int)((long long)all * (s + 1) / splits))) {
        const size_t at = ((size_t)s * p.heads + head) * p.T + row;
        ml[s] = p.ml[at];
        o[s] = __ldcs(reinterpret_cast<const float4*>(p.part + at * p.dv) + v);
      }
    }
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s) ref = fmaxf(ref, ml[s].x);
    ref = ref == -INFINITY ? 0.0f : ref;
    float l = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s) {
      if (ml[s].x == -INFINITY && ml[s].y == 0.0f) continue;   // the row saw none of the share's tokens
      const float w = ex2(ml[s].x - ref);
      l = fmaf(w, ml[s].y, l);
      acc.x = fmaf(w, o[s].x, acc.x);
      acc.y = fmaf(w, o[s].y, acc.y);
      acc.z = fmaf(w, o[s].z, acc.z);
      acc.w = fmaf(w, o[s].w, acc.w);
    }
    uint2 packed;
    packed.x = bf16x2_of(acc.x / l, acc.y / l);
    packed.y = bf16x2_of(acc.z / l, acc.w / l);
    reinterpret_cast<uint2*>(p.out + (row * p.heads + head) * p.dv)[v] = packed;
  }
}

// ---------------------------------------------------------------- host side
struct PrefillWs {
  size_t counts, blocks, tiles, k, v, r, part, ml, bytes;
  int rows, n_blocks, splits;
};

bool prefill_shape_ok(int B, int T, int heads, int dn, int dv, int kv_tokens) {
  if ((dn != 64 && dn != 128) || (dv != 64 && dv != 128) || heads > 1024 || B > kMaxB) return false;
  return (long long)T * heads <= INT_MAX && ((long long)kv_tokens + 128LL * B) * heads <= INT_MAX;
}

// Shares of a block's tokens that a call has room for: up to about two items per SM (the plan takes what pays).  From
// the queries' number alone, so that a loose kv_tokens changes no result.
int most_shares(long long items) {
  const long long s = 2LL * num_sms() / items;
  return s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : (int)s;
}

// Rows of partial results that there is room for: the most that a call of up to T queries and any number of sequences
// writes.  Fewer queries can mean more shares, so the room for T alone would not do for the short last chunk of a prompt.
size_t share_rows(int T, int heads) {
  size_t most = 0;
  for (int s = 2; s <= kMaxSplits; ++s) {
    const long long blocks = 2LL * num_sms() / ((long long)heads * s);   // T / kBlock + 1 at most, for s shares or more
    if (blocks < 1) continue;
    const long long t = kBlock * blocks - 1;
    const size_t rows = (size_t)s * (size_t)(t < T ? t : T);
    if (rows > most) most = rows;
  }
  return most;
}

PrefillWs prefill_ws(int B, int T, int heads, int dn, int dv, int rope, int kv_tokens) {
  PrefillWs w;
  w.rows = (kv_tokens + kRowAlign - 1) / kRowAlign * kRowAlign + kRowAlign * (B - 1);
  w.n_blocks = T / kBlock + B;
  size_t at = 0;
  w.counts = at;
  at += 256;
  w.blocks = at;
  at += align_up((size_t)w.n_blocks * sizeof(QBlock), 256);
  w.tiles = at;
  at += align_up((size_t)(w.rows / kRowAlign) * sizeof(TokTile), 256);
  w.k = at;
  at += align_up((size_t)heads * w.rows * dn * 2, 256);
  w.v = at;
  at += align_up((size_t)heads * w.rows * dv * 2, 256);
  w.r = at;
  at += align_up((size_t)w.rows * (rope ? rope : 8) * 2, 256);
  w.splits = most_shares((long long)w.n_blocks * heads);
  w.part = at;
  const size_t shares = share_rows(T, heads) * heads;
  at += align_up(shares * dv * sizeof(float), 256);
  w.ml = at;
  at += align_up(shares * sizeof(float2), 256);
  w.bytes = at;
  return w;
}

template <int KC, int VC>
cudaError_t launch_attend(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mr, const CUtensorMap& mv,
                          const PrefillParams& p, cudaStream_t s) {
  using A = Attend<KC>;
  static_assert(A::kSmem + sizeof(Shared) <= 227 * 1024, "shared memory");
  static std::atomic<unsigned char> attr[kMaxDevices];
  const cudaError_t e = once_per_device(attr, [] {
    return cudaFuncSetAttribute(attend_kernel<KC, VC>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::kSmem);
  });
  return e == cudaSuccess ? launch_k(attend_kernel<KC, VC>, num_sms(), kThreads, A::kSmem, s, mq, mk, mr, mv, p) : e;
}

// f16 bits move like bf16 bits: the maps' element type only has to be 16 bits wide
int launch_prefill(const PrefillParams& p, cudaStream_t s) {
  CUtensorMap mq, mk, mr, mv, mx, mw;
  const uint64_t rows = (uint64_t)p.heads * p.kv_rows;
  const uint64_t cache_rows = (uint64_t)p.kv.n_layers * p.kv.n_pages * p.kv.page_tokens;
  if (!make_map(&mq, p.q, (uint64_t)p.heads * (p.dn + p.rope), p.T, kTile) || !make_map(&mk, p.k, p.dn, rows, kTile) ||
      !make_map(&mr, p.rope ? (void*)p.r : (void*)p.k, p.rope ? p.rope : p.dn, p.rope ? p.kv_rows : rows, kTile) ||
      !make_map(&mv, p.v, p.dv, rows, kTile) || !make_map(&mx, p.kv.pages, p.kv.row, cache_rows, p.kv.page_tokens) ||
      !make_map(&mw, p.w, p.kv.rank, (uint64_t)p.heads * (p.dn + p.dv), p.dn + p.dv))
    return MOE_ERR_CUDA;
  const int ex_smem = p.kv.rank / kBK * kChunkBytes + kExStages * kExStage + 1024;
  constexpr int kExSmem = kMaxChunks * kChunkBytes + kExStages * kExStage + 1024;
  static_assert(kExSmem + sizeof(ExShared) <= 227 * 1024, "shared memory");
  static std::atomic<unsigned char> attr[kMaxDevices];
  cudaError_t e = once_per_device(attr, [] {
    return cudaFuncSetAttribute(expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExSmem);
  });
  if (e == cudaSuccess && p.B > kSmallB) e = launch_k(plan_kernel, 1, kPlanThreads, 0, s, p);
  if (e == cudaSuccess) e = launch_k(expand_kernel, num_sms(), kExThreads, ex_smem, s, mx, mw, p);
  if (e == cudaSuccess) {
    const int kc = p.dn / kBK + (p.rope ? 1 : 0), vc = p.dv / kBK;
    e = vc == 2 ? (kc == 3   ? launch_attend<3, 2>(mq, mk, mr, mv, p, s)
                   : kc == 2 ? launch_attend<2, 2>(mq, mk, mr, mv, p, s)
                             : launch_attend<1, 2>(mq, mk, mr, mv, p, s))
                : (kc == 3   ? launch_attend<3, 1>(mq, mk, mr, mv, p, s)
                   : kc == 2 ? launch_attend<2, 1>(mq, mk, mr, mv, p, s)
                             : launch_attend<1, 1>(mq, mk, mr, mv, p, s));
  }
  if (e == cudaSuccess && p.max_splits > 1)
    e = launch_k(combine_splits_kernel, dim3(p.max_blocks_q, 8 * num_sms() / p.max_blocks_q + 1), 256, 0, s, p);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_latent_prefill_workspace_size(const moe_kv_cache* cache, int B, int T, int heads, int dn, int dv,
                                         int kv_tokens) {
  if (check_latent(cache, 0) != MOE_OK || B < 1 || T < 1 || heads < 1 || kv_tokens < 1) return 0;
  return prefill_shape_ok(B, T, heads, dn, dv, kv_tokens) ? prefill_ws(B, T, heads, dn, dv, cache->rope, kv_tokens).bytes : 0;
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
  if (!kv_aligned(q, 16) || !kv_aligned(w_kv, 16) || !kv_aligned(out, 32)) return MOE_ERR_UNSUPPORTED;
  const PrefillWs w = prefill_ws(B, T, heads, dn, dv, cache->rope, kv_tokens);
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
  p.rope = cache->rope;
  p.kv_rows = w.rows;
  p.max_blocks_q = w.n_blocks;
  // zero as the smallest normal number: a token out of sight scores -infinity, and 0 * -infinity is NaN
  p.scale_log2 = scale == 0.0f ? FLT_MIN : scale * 1.4426950408889634f;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.seqs = seqs;
  p.q_off = q_offsets;
  p.w = reinterpret_cast<const __nv_bfloat16*>(w_kv);
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.counts = reinterpret_cast<int32_t*>(b + w.counts);
  p.blocks = reinterpret_cast<QBlock*>(b + w.blocks);
  p.tiles = reinterpret_cast<TokTile*>(b + w.tiles);
  p.k = reinterpret_cast<__nv_bfloat16*>(b + w.k);
  p.v = reinterpret_cast<__half*>(b + w.v);
  p.r = reinterpret_cast<__nv_bfloat16*>(b + w.r);
  p.max_splits = w.splits;
  p.sms = num_sms();
  p.part = reinterpret_cast<float*>(b + w.part);
  p.ml = reinterpret_cast<float2*>(b + w.ml);
  p.status = dev_status;
  return launch_prefill(p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
