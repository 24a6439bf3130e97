// What the queries of an absorbed latent attention looked at: per cached token
// the sum of its probabilities over all query rows, from the log-sum-exp that the
// attention left.
//
// A tile is 128 tokens against up to 128 query rows (a row = one query token of one head):
//   S = K Q^T     M = tokens (128), N = query rows, K = rank + rope
//   w[t] += sum_r exp(S[t, r] - lse[r])
// Tokens are M, so that a token's sum is one thread's: no exchange between
// threads, no atomics, the rows always in the same order.
//
// Work: the sequences' tokens form one line, in units of 32, that is cut evenly
// over the CTAs; a tile is up to four units of one sequence.  Up to 64 query rows
// stay in shared memory while their sequence's tiles pass by; more come in passes of
// up to 128, in 64-entry chunks that stream through a ring once per tile, each CTA
// beginning with another pass (all at once on the same rows, they wait for the few
// L2 slices that hold them).  Where there are fewer units than CTAs, a unit's passes
// are shared out, and finish_weights_kernel adds the shares in order.
//
// Bound: the rows of the cache, read once (bf16: 6.6 TB/s on long batches), in 4
// bits their expansion (about 7500 cycles a tile), with many query rows the products
// (a pass of 128 takes 2304 cycles of them, and 5000 with what lies between its parts).
// Measured, rank 512 and rope 64:
//   32 x 250..6001, 64 heads             23.6 us   4.3 TB/s; 832,000 tokens (967 MB with their weights) 147 us
//   32 x 250..6001, 64 heads, 4 bits     28 us     832,000 tokens 167 us
//   1 x 16001, 32 queries of 32 heads    28.7 us   4 bits 30.5
//
// Roles: warp 0 = copies of the cache, warp 1 = products (and TMEM owner), warp 2 =
// copies of the queries, warps 4..7 = sums, and for a cache in 4 bits warps 8..15, which
// expand its rows.  Every mbarrier wait is bounded; on expiry the CTA reports
// MOE_DEV_ERR_TIMEOUT, drains and returns.
#include <cfloat>
#include <cmath>

#include "kv_fp4.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kTile = 128;                       // tokens
constexpr int kUnit = 32;                        // tokens that the line is cut by
constexpr int kChunkBytes = kTile * kBK * 2;     // 16 KB: 128 rows x 64 entries
constexpr int kMaxPairs = 4;                     // 128-entry slices of the latent
constexpr int kMaxParts = kMaxPairs + 1;         // and the rotary key
constexpr int kResident = 64;                    // query rows that stay in shared memory
constexpr int kPassRows = 128;                   // query rows of a pass where they do not
constexpr int kRing = 2;                         // parts of such a pass in flight
constexpr int kThreads = 256;                    // a bf16 cache's; one in 4 bits has kExpandWarps more
constexpr int kExpandWarps = 8;
constexpr int kSumThreads = 128;
constexpr int kTmemCols = 256;                   // two passes of 128 columns
constexpr int kBatch = 256;                      // sequences of one launch: their lengths lie in shared memory, and 256 times 2^27
                                                 // tokens are 2^30 units
constexpr float kLog2e = 1.4426950408889634f;

struct WeightParams {
  KvView kv;
  int layer, B, Q, heads, first;      // first: the launch's first entry of the list
  int pairs, parts;                   // a row comes in parts: 128-entry pairs of chunks, then the rotary key
  int passes, rows_pass, ring;        // passes over the query rows, rows of each, parts of queries in shared memory
  int ctas;
  bool resident;                      // the queries stay in shared memory while their sequence's tiles pass by
  float scale_log2, decay;
  const int32_t* seqs;                // the whole list
  const float* lse;
  float* weights;
  int32_t* plan;                      // [B + 1] units before each sequence
  float* part;                        // [ctas][32] sums of a unit's shares
  uint32_t* status;
};

// A tile of one sequence, and which of the passes over its query rows.
struct Tile {
  int b, seq, t0, t1, len, work, p0, p1;
  bool first, last;    // of its sequence in this CTA
};

// Shares of a unit's passes.
__host__ __device__ inline int pass_shares(int units, int passes, int ctas) {
  const int s = units > 0 ? ctas / units : 1;
  return s < 1 ? 1 : s < passes ? s : passes;
}

struct Tiles {
  const int *pref, *len, *ids;
  int u, u1, b, shares, share, p0, p1;

  __device__ Tiles(const WeightParams& p, const int* pref_, const int* len_, const int* ids_) : pref(pref_), len(len_), ids(ids_) {
    const int units = pref[p.B];
    shares = pass_shares(units, p.passes, p.ctas);
    const int per = (units + p.ctas - 1) / p.ctas;      // 1 where units are shared out
    u = (int)min((long long)units, (long long)(blockIdx.x / shares) * per);
    u1 = min(units, u + per);
    share = blockIdx.x % shares;
    p0 = p.passes * share / shares;
    p1 = p.passes * (share + 1) / shares;
    int lo = 0, hi = p.B;   // the last b with pref[b] <= the first unit
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pref[mid] <= u) lo = mid;
      else hi = mid;
    }
    b = lo;
    first = true;
  }
  __device__ bool next(Tile& t) {
    if (u >= u1) return false;
    while (pref[b + 1] <= u) {
      ++b;
      first = true;
    }
    const int end = min(pref[b + 1], u1), n = min(kTile / kUnit, end - u);
    t.b = b;
    t.seq = ids[b];
    t.len = len[b];
    t.t0 = (u - pref[b]) * kUnit;
    t.t1 = min(t.len, t.t0 + n * kUnit);
    t.work = u * shares + share;
    t.p0 = p0;
    t.p1 = p1;
    t.first = first;
    t.last = u + n >= end;
    first = false;
    u += n;
    return true;
  }
  // the k-th pass of a tile
  __device__ static int pass(const Tile& t, int k) { return t.p0 + (k + (int)blockIdx.x) % (t.p1 - t.p0); }

 private:
  bool first;
};

struct alignas(16) Shared {
  uint64_t k_full[kMaxParts], k_empty[kMaxParts], q_full[kMaxParts], q_empty[kMaxParts], d_full[2], d_empty[2], drain;
  uint32_t tmem;
  int abort;
  int warp_sum[kThreads / 32 + kExpandWarps];
  int repeat;
  union {
    uint32_t listed[kMaxSeqs / 32];               // bit by bit: ids met so far
    struct {
      alignas(16) float lse[2][kPassRows];        // read four at a time: of a pass's rows, times log2(e)
      alignas(16) int limit[2][kPassRows];        // the tokens below it are seen by the row
    };
  };
  int pref[kBatch + 1];
  int len[kBatch];
  int ids[kBatch];
};

// All threads of the sums' warps (named barrier 1).
__device__ inline void sums_meet() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kSumThreads) : "memory");
}

// 32 columns' probabilities of one token.  `edge`: rows that do not see it, or columns past the pass's rows.
__device__ inline float sum32(const uint32_t (&s)[32], const float* lse, const int* limit, int t, int rows, float scale, bool edge) {
  float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int x = 0; x < 32; x += 4) {
    const float4 l = *reinterpret_cast<const float4*>(lse + x);
    float e[4] = {ex2(fmaf(__uint_as_float(s[x]), scale, -l.x)), ex2(fmaf(__uint_as_float(s[x + 1]), scale, -l.y)),
                  ex2(fmaf(__uint_as_float(s[x + 2]), scale, -l.z)), ex2(fmaf(__uint_as_float(s[x + 3]), scale, -l.w))};
    if (edge) {
      const int4 m = *reinterpret_cast<const int4*>(limit + x);
      e[0] = (t < m.x) & (x < rows) ? e[0] : 0.0f;
      e[1] = (t < m.y) & (x + 1 < rows) ? e[1] : 0.0f;
      e[2] = (t < m.z) & (x + 2 < rows) ? e[2] : 0.0f;
      e[3] = (t < m.w) & (x + 3 < rows) ? e[3] : 0.0f;
    }
    a = add2(a, add2(make_float2(e[0], e[1]), make_float2(e[2], e[3])));
  }
  return a.x + a.y;
}

template <bool FP4>
__global__ void __launch_bounds__(kThreads + (FP4 ? 32 * kExpandWarps : 0), 1)
weights_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_q, const WeightParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kAll = kThreads + (FP4 ? 32 * kExpandWarps : 0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int j = 0; j < kMaxParts; ++j) {
      mbar_init(&sh.k_full[j], FP4 && j < p.pairs ? kExpandWarps : 1);
      mbar_init(&sh.k_empty[j], 1);
      mbar_init(&sh.q_full[j], 1);
      mbar_init(&sh.q_empty[j], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.d_full[i], 1);
      mbar_init(&sh.d_empty[i], kSumThreads / 32);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    sh.repeat = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 96) {
    prefetch_map(&map_k);
    prefetch_map(&map_q);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  for (int i = tid; i < kMaxSeqs / 32; i += kAll) sh.listed[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // Ids, and whether any of them was listed before (in this launch's part of the list or an earlier one's).
  for (int i = tid; i < p.first + p.B; i += kAll) {
    const int s = p.seqs[i];
    if (i >= p.first) sh.ids[i - p.first] = s;
    if (s >= 0 && s < p.kv.max_seqs && (atomicOr(&sh.listed[s >> 5], 1u << (s & 31)) >> (s & 31) & 1u)) sh.repeat = 1;
  }
  __syncthreads();
  const bool repeat = sh.repeat != 0;
  {
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAll) {
      const int b = b0 + tid;
      int n = 0;
      if (b < p.B) {
        const int s = sh.ids[b];
        bool good = s >= 0 && s < p.kv.max_seqs;
        if (good && repeat)      // rare: look for the entry's first place
          for (int j = 0; good && j < p.first + b; ++j) good = p.seqs[j] != s;
        if (!good && blockIdx.x == 0) set_status(p.status, MOE_DEV_ERR_BAD_SEQ);
        const int len = good ? p.kv.len_of(s) : 0;
        sh.len[b] = len;
        n = (len + kUnit - 1) / kUnit;
      }
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      if (lane == 31) sh.warp_sum[warp] = inc;
      __syncthreads();
      int base = carry;
      for (int w = 0; w < warp; ++w) base += sh.warp_sum[w];
      for (int w = 0; w < kAll / 32; ++w) carry += sh.warp_sum[w];
      if (b < p.B) sh.pref[b + 1] = base + inc;
      __syncthreads();
    }
    if (tid == 0) sh.pref[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.B; b += kAll) p.plan[b] = sh.pref[b];
  const uint32_t tmem = sh.tmem;
  volatile int* abort_flag = &sh.abort;
  const int rows_all = p.Q * p.heads, q_chunk = p.rows_pass * 128;
  uint8_t* sq = smem + (2 * p.pairs + (p.parts > p.pairs)) * kChunkBytes;
  Tiles it(p, sh.pref, sh.len, sh.ids);
  Tile tl;

  if (warp == 0) {
    // ------------------------------------------------ copies of the cache (in 4 bits: of the rotary keys)
    const int page = p.kv.page_tokens, box = min(page, kUnit), layer_page = p.layer * p.kv.n_pages;
    const uint32_t smem0 = uni(smem_u32(smem)), bar0 = uni(smem_u32(&sh.k_full[0]));
    const uint64_t once = l2_evict_first();
    const int j_first = FP4 ? p.pairs : 0;
    int tile = 0;
    bool ok = true;
    while (__any_sync(0xffffffffu, ok && it.next(tl))) {
      const int nb = (int)uni((tl.t1 - tl.t0 + box - 1) / box);
      int row = 0;
      if (lane < nb) {
        const int t = tl.t0 + lane * box;
        int pg = p.kv.table[(size_t)tl.seq * p.kv.max_blocks + (t >> p.kv.page_shift)];
        if (pg < 0 || pg >= p.kv.n_pages) {
          set_status(p.status, MOE_DEV_ERR_BAD_PAGE);
          pg = 0;
        }
        row = (layer_page + pg) * page + (t & (page - 1));
      }
      int rows[kTile / 16];
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i) rows[i] = (int)uni(lane == i ? row : 0);
      for (int j = j_first; j < p.parts; ++j) {
        ok = warp_wait(&sh.k_empty[j], (tile & 1) ^ 1u, abort_flag);
        if (!ok) break;
        const bool pair = j < p.pairs;
        const uint32_t to = smem0 + 2 * j * kChunkBytes, bar = bar0 + 8 * j;
        const int at = pair ? 2 * j * kBK : p.kv.rope_at;
        mbar_expect_tx_warp(bar, (uint32_t)(nb * box * (pair ? 256 : 128)));
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
          if (i < nb) {
            tma_load_2d_hint_warp(to + i * box * 128, &map_k, bar, at, rows[i], once);
            if (pair) tma_load_2d_hint_warp(to + kChunkBytes + i * box * 128, &map_k, bar, at + kBK, rows[i], once);
          }
      }
      ++tile;
    }
    // drain: whatever was asked for lands before the CTA can exit
    volatile int no_abort = 0;
    if (tile)
      for (int j = j_first; j < p.parts; ++j) mbar_wait(&sh.k_full[j], (tile - 1) & 1, &no_abort);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------ copies of the queries
    const uint32_t q0 = uni(smem_u32(sq)), bar0 = uni(smem_u32(&sh.q_full[0]));
    const uint64_t keep = l2_normal();
    int slot = 0, loads = 0;
    uint32_t par = 1;
    bool ok = true;
    while (__any_sync(0xffffffffu, ok && it.next(tl))) {
      if (p.resident && !tl.first) continue;               // they are there
      const int n = (int)uni(tl.p1 - tl.p0);
      for (int k = 0; ok && k < n; ++k) {
        const int row0 = (int)uni(tl.b * rows_all + Tiles::pass(tl, k) * p.rows_pass);
        for (int j = 0; j < p.parts; ++j) {
          ok = warp_wait(&sh.q_empty[slot], par, abort_flag);
          if (!ok) break;
          const bool pair = j < p.pairs;
          const uint32_t to = q0 + 2 * slot * q_chunk, bar = bar0 + 8 * slot;
          mbar_expect_tx_warp(bar, (uint32_t)(pair ? 2 * q_chunk : q_chunk));
          tma_load_2d_hint_warp(to, &map_q, bar, 2 * j * kBK, row0, keep);      // the rotary key stands behind the latent
          if (pair) tma_load_2d_hint_warp(to + q_chunk, &map_q, bar, 2 * j * kBK + kBK, row0, keep);
          ++loads;
          if (++slot == p.ring) {
            slot = 0;
            par ^= 1u;
          }
        }
      }
    }
    volatile int no_abort = 0;
    for (int s = 0; s < p.ring; ++s) {
      const int n = loads / p.ring + (loads % p.ring > s ? 1 : 0);
      if (n > 0) mbar_wait(&sh.q_full[s], (n - 1) & 1, &no_abort);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ products
    const uint32_t tm = uni(tmem), smem0 = uni(smem_u32(smem));
    const uint32_t sq0 = uni(smem_u32(sq));
    const uint64_t dk0 = smem_desc(smem0), dq0 = smem_desc(sq0), q_step = (uint64_t)(q_chunk >> 4);
    int tile = 0, pass = 0, slot = 0;
    uint32_t par = 0;
    bool ok = true, issued = false;
    while (__any_sync(0xffffffffu, ok && it.next(tl))) {
      const int n = (int)uni(tl.p1 - tl.p0);
      const bool keep = p.resident && !uni(tl.last);        // the next tile takes the same queries
      for (int k = 0; ok && k < n; ++k, ++pass) {
        const int buf = pass & 1, g = (int)uni(Tiles::pass(tl, k));
        ok = warp_wait(&sh.d_empty[buf], ((pass >> 1) & 1) ^ 1u, abort_flag);
        if (!ok) break;
        const uint32_t idesc = make_idesc(kTile, (min(p.rows_pass, rows_all - g * p.rows_pass) + 15) & ~15);
        const uint32_t d = tm + buf * kPassRows;
        for (int j = 0; j < p.parts; ++j) {
          ok = warp_wait(&sh.q_full[slot], par, abort_flag) && warp_wait(&sh.k_full[j], tile & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dk = dk0 + ((uint64_t)(2 * j * kChunkBytes) >> 4), dq = dq0 + 2 * slot * q_step;
          if (j < p.pairs) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              tc_mma_warp(d, dk + (((x >> 2) * kChunkBytes + (x & 3) * kUK * 2) >> 4),
                          dq + ((x & 3) * kUK * 2 >> 4) + (x >> 2) * q_step, idesc, x ? 1u : (j ? 1u : 0u));
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (x * kUK < p.kv.rope) tc_mma_warp(d, dk + ((x * kUK * 2) >> 4), dq + ((x * kUK * 2) >> 4), idesc, 1u);
          }
          issued = true;
          if (k == n - 1) tc_commit_warp(&sh.k_empty[j]);
          if (!keep) tc_commit_warp(&sh.q_empty[slot]);
          if (++slot == p.ring) {
            slot = 0;
            if (!keep) par ^= 1u;
          }
        }
        if (ok) tc_commit_warp(&sh.d_full[buf]);
      }
      ++tile;
    }
    if (issued) {   // every issued product completes before tensor memory is released
      volatile int no_abort = 0;
      tc_commit_warp(&sh.drain);
      mbar_wait(&sh.drain, 0, &no_abort);
    }
    __syncwarp();
  } else if (FP4 && warp >= kThreads / 32) {
    // ------------------------------------------------ latents in 4 bits, expanded into the tile that a copy would fill
    // Four threads a token, two tokens a thread; of each 128-entry pair a thread has 16 bytes of codes, a quarter.  Codes
    // are asked for a pair ahead, pages a tile ahead.  Places past a tile's last token get some row's entries: the sums
    // there are not written.
    const int r = (warp - kThreads / 32) * 8 + (lane & 7), v = lane >> 3;
    const int scales_at = p.kv.rank / 2 + 2 * p.kv.rope;
    const Fp4Place to(smem_u32(smem), kChunkBytes, r, v);      // of the first token; the second's lies 64 rows on
    const uint8_t* row[2];
    int page[2], at[2];           // of the next tile: page and place in it
    uint4 code[2];
    uint32_t scale[2];
    int j_load = 0;
    auto look_up = [&](bool any) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = tl.t0 + r + 64 * e;
        page[e] = at[e] = 0;
        if (any && t < tl.t1) {
          page[e] = __ldg(p.kv.table + (size_t)tl.seq * p.kv.max_blocks + (t >> p.kv.page_shift));
          at[e] = t & (p.kv.page_tokens - 1);
        }
      }
    };
    auto locate = [&]() {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (page[e] < 0 || page[e] >= p.kv.n_pages) {
          set_status(p.status, MOE_DEV_ERR_BAD_PAGE);
          page[e] = 0;
        }
        row[e] = reinterpret_cast<const uint8_t*>(p.kv.pages + p.kv.row_offset(p.layer, page[e], at[e])) + 16 * v;
      }
    };
    auto load = [&](int e) {
      code[e] = ldg_stream(row[e] + 64 * j_load);
      scale[e] = ldg_stream_u16(row[e] + scales_at + 8 * j_load - 14 * v);
    };
    bool now = it.next(tl), ok = true;
    look_up(now);
    locate();
    load(0);
    load(1);
#pragma unroll 1
    for (int tile = 0; ok && now; ++tile) {
      const bool next = it.next(tl);
      look_up(next);
#pragma unroll 1
      for (int j = 0; j < p.pairs; ++j) {
        if (++j_load == p.pairs) {
          j_load = 0;
          locate();
        }
        ok = warp_wait(&sh.k_empty[j], (tile & 1) ^ 1u, abort_flag);
        if (!ok) break;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          fp4_store32<2>(to, 2 * j * kChunkBytes + e * (64 * 128), code[e], scale[e]);
          load(e);
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.k_full[j]);
      }
      now = next;
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------ sums: a thread a token
    const int quarter = warp & 3, st = tid - kSumThreads;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const size_t cap = (size_t)p.kv.max_blocks << p.kv.page_shift;
    const float scale = p.scale_log2;
    int pass = 0, stage = 0;
    bool ok = true;
    while (it.next(tl)) {
      const int t = tl.t0 + st;
      float* w = p.weights + (size_t)tl.seq * cap + t;
      const bool mine = t < tl.t1;
      const float old = mine && it.shares == 1 && p.decay != 0.0f ? *w : 0.0f;
      float sum = 0.0f;
      // a thread brings one row's log-sum-exp, a pass ahead
      const float* lse = p.lse + (size_t)(p.first + tl.b) * rows_all;
      auto lse_of = [&](int k) {
        const int r = Tiles::pass(tl, k) * p.rows_pass + st;
        const float x = st < p.rows_pass && r < rows_all ? lse[r] * kLog2e : 0.0f;
        return x == -INFINITY ? INFINITY : x;       // a row that looked at nothing adds nothing: s - infinity, not s + infinity
      };
      float ahead = p.passes > 1 || tl.first ? lse_of(0) : 0.0f;
      const int n = tl.p1 - tl.p0;
      for (int k = 0; k < n; ++k, ++pass) {
        const int g = Tiles::pass(tl, k);
        const int rows = min(p.rows_pass, rows_all - g * p.rows_pass);
        if (p.passes > 1 || tl.first) {
          stage ^= 1;
          if (st < rows) {
            sh.lse[stage][st] = ahead;
            sh.limit[stage][st] = tl.len - p.Q + (g * p.rows_pass + st) / p.heads + 1;
          }
          if (k + 1 < n) ahead = lse_of(k + 1);
          sums_meet();      // whoever writes this stage's place next has met everyone who read it
        }
        const int buf = pass & 1;
        // a warp whose wait ran out goes on through the passes without their sums: the others wait for it at sums_meet
        if (!warp_wait(&sh.d_full[buf], (pass >> 1) & 1, abort_flag)) {
          ok = false;
          continue;
        }
        tc_fence_after();
        const int limit0 = tl.len - p.Q + g * p.rows_pass / p.heads + 1;       // the pass's first row sees the least
        const bool seen = tl.t1 <= limit0;
        for (int c = 0; c < rows; c += 32) {
          uint32_t s[32];
          tmem_ld32(lane_base + buf * kPassRows + c, s);
          tmem_ld_wait();
          const float* l = sh.lse[stage] + c;
          const int* limit = sh.limit[stage] + c;
          sum += seen && c + 32 <= rows ? sum32(s, l, limit, t, rows - c, scale, false) : sum32(s, l, limit, t, rows - c, scale, true);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.d_empty[buf]);
      }
      if (!ok) continue;
      if (it.shares > 1) {
        if (st < kUnit) p.part[(size_t)tl.work * kUnit + st] = sum;
      } else if (mine) {
        *w = p.decay == 0.0f ? sum : fmaf(p.decay, old, sum);
      }
    }
  }
  __syncthreads();
  if (*abort_flag && tid == 0) set_status(p.status, MOE_DEV_ERR_TIMEOUT);
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// Shares of units, added in order (calls of more than one pass; returns at once where none were shared out).
__global__ void __launch_bounds__(kUnit) finish_weights_kernel(const WeightParams p) {
  pdl_wait();
  pdl_trigger();
  const int units = p.plan[p.B], shares = pass_shares(units, p.passes, p.ctas), unit = blockIdx.x;
  if (shares == 1 || unit >= units) return;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.plan[mid] <= unit) lo = mid;
    else hi = mid;
  }
  const int seq = p.seqs[p.first + lo], t = (unit - p.plan[lo]) * kUnit + threadIdx.x;
  if (t >= p.kv.len_of(seq)) return;
  float sum = 0.0f;
  for (int s = 0; s < shares; ++s) sum += p.part[((size_t)unit * shares + s) * kUnit + threadIdx.x];
  float* w = p.weights + (size_t)seq * ((size_t)p.kv.max_blocks << p.kv.page_shift) + t;
  *w = p.decay == 0.0f ? sum : fmaf(p.decay, *w, sum);
}

// ---------------------------------------------------------------- host side
bool weights_shape_ok(int B, int Q, int heads) { return B <= 4096 && (long long)Q * heads <= 1024; }

size_t plan_bytes(int B) { return align_up((size_t)((B < kBatch ? B : kBatch) + 1) * sizeof(int32_t), 256); }

template <bool FP4>
cudaError_t launch_weights(const CUtensorMap& mk, const CUtensorMap& mq, const WeightParams& p, int smem, cudaStream_t s) {
  static std::atomic<unsigned char> attr[kMaxDevices];
  const cudaError_t e = once_per_device(attr, [] {
    return cudaFuncSetAttribute(weights_kernel<FP4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                227 * 1024 - (int)sizeof(Shared));
  });
  constexpr int threads = kThreads + (FP4 ? 32 * kExpandWarps : 0);
  return e == cudaSuccess ? launch_k(weights_kernel<FP4>, p.ctas, threads, smem, s, mk, mq, p) : e;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_latent_weights_workspace_size(const moe_kv_cache* cache, int B, int Q, int heads) {
  if (check_latent(cache, 0) != MOE_OK || B < 1 || Q < 1 || heads < 1 || !weights_shape_ok(B, Q, heads)) return 0;
  return plan_bytes(B) + (Q * heads > kResident ? align_up((size_t)num_sms() * kUnit * sizeof(float), 256) : 0);
}

int moe_latent_weights(const moe_kv_cache* cache, int layer, const void* q, const int32_t* seqs, int B, int Q, int heads,
                       float scale, const float* lse, float decay, float* weights, void* ws, size_t ws_bytes,
                       uint32_t* dev_status, moe_stream_t stream) {
  constexpr int kMaxChunks = 2 * kMaxPairs + 1;
  static_assert(sizeof(Shared) + 1024 + kMaxChunks * (kChunkBytes + kResident * kBK * 2) <= 227 * 1024 &&
                    2 * kRing * kPassRows <= kMaxChunks * kResident, "shared memory");
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
  const bool fp4 = cache->format == MOE_KV_FP4;
  const int rows = Q * heads, row = cache->rank + cache->rope;
  WeightParams p;
  p.kv = kv_view(*cache);
  p.layer = layer;
  p.Q = Q;
  p.heads = heads;
  p.pairs = cache->rank / 128;
  p.parts = p.pairs + (cache->rope ? 1 : 0);
  const int most = rows <= kResident ? kResident : kPassRows;
  p.passes = (rows + most - 1) / most;
  p.rows_pass = ((rows + p.passes - 1) / p.passes + 15) & ~15;       // evenly, in multiples of 16
  p.passes = (rows + p.rows_pass - 1) / p.rows_pass;
  p.resident = rows <= kResident;
  p.ring = p.resident ? p.parts : kRing;
  p.ctas = num_sms();
  // zero as the smallest normal number, as in the attention whose log-sum-exp this is
  p.scale_log2 = scale == 0.0f ? FLT_MIN : scale * kLog2e;
  p.decay = decay;
  p.seqs = seqs;
  p.lse = lse;
  p.weights = weights;
  p.plan = reinterpret_cast<int32_t*>(ws);
  p.part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + plan_bytes(B));
  p.status = dev_status;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int chunks = 2 * p.pairs + (cache->rope ? 1 : 0), q_chunks = p.resident ? chunks : 2 * kRing;
  const int smem = chunks * kChunkBytes + q_chunks * p.rows_pass * kBK * 2 + 1024;
  CUtensorMap mk;
  if (!make_map(&mk, cache->pages, p.kv.row, (uint64_t)cache->n_layers * cache->n_pages * cache->page_tokens,
                cache->page_tokens < kUnit ? cache->page_tokens : kUnit))
    return MOE_ERR_CUDA;
  for (int b0 = 0; b0 < B; b0 += kBatch) {   // longer lists: several launches
    p.first = b0;
    p.B = B - b0 < kBatch ? B - b0 : kBatch;
    CUtensorMap mq;
    if (!make_map(&mq, reinterpret_cast<const __nv_bfloat16*>(q) + (size_t)b0 * rows * row, row, (uint64_t)p.B * rows, p.rows_pass))
      return MOE_ERR_CUDA;
    cudaError_t e = fp4 ? launch_weights<true>(mk, mq, p, smem, s) : launch_weights<false>(mk, mq, p, smem, s);
    if (e == cudaSuccess && p.passes > 1) e = launch_k(finish_weights_kernel, p.ctas / 2, kUnit, 0, s, p);   // no more units are shared out
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
