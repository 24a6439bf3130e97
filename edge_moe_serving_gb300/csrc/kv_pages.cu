// Pages of the latent cache: reserving, storing rows, forking, freeing and
// compacting.  All state is on the device and every choice is a function of it
// (lowest free page first, list order), so the calls can be captured and give
// the same tables on every run.
//
// A call that takes or moves pages is two steps: one CTA plans (a scan over
// refs, 4096 pages a round, that stops once it has what it needs), then the plan
// is applied, by the whole grid or, for small calls, by a cluster in the same
// launch: tables and reference counts by integer adds, which commute, and page
// rows by 16-byte copies.  Bound: the rows that move, read and written once; for
// small calls on pools of a few rounds the plan's dependent reads and the launches.
// 16 beams that change parents: 6.5 us.  64 branches off 8 contexts, 4 layers, 14.9
// MB: 8.2 us.  A quarter of 64 sequences replaced, 4 layers, 968 MB: 163 us, 5.9 TB/s.
// One token more for 64 sequences, 4 layers (a reserve and four appends): 12.0 us.
// On large pools the scan is what counts, about 0.9 us a round: with the free pages
// behind all others a reserve of 64 pages takes 5 us of 1,000 and 4,000 pages, 7 of
// 16,000, 19 of 64,000 and 33 of 128,000; a compaction that moves nothing 4, 4, 9, 26
// and 49 (two rounds each).
#include "kv_append_shape.h"
#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 256;
constexpr int kCluster = 8;              // CTAs of the one-launch forms

// All threads of the cluster's CTAs; what they wrote before is seen after.
__device__ inline void cluster_meet() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct PlanScan {
  int warp[32];
  int total;
};

// Exclusive prefix sum over the CTA's threads; `total` gets the sum.
__device__ inline int cta_scan(int v, PlanScan& sh, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) sh.warp[w] = inc;
  __syncthreads();
  if (w == 0) {
    int s = lane < (int)(blockDim.x >> 5) ? sh.warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    sh.warp[lane] = s;
    if (lane == 31) sh.total = s;
  }
  __syncthreads();
  const int base = w ? sh.warp[w - 1] : 0;
  total = sh.total;
  __syncthreads();
  return base + inc - v;
}

// The `want` lowest free pages, ascending, into list[]; returns how many there are (at most want).
__device__ int lowest_free(const KvView& kv, int want, int32_t* list, PlanScan& sh) {
  int found = 0;
  for (int p0 = 0; p0 < kv.n_pages && found < want; p0 += 4 * kPlanThreads) {
    const int p = p0 + 4 * threadIdx.x;
    bool f[4];
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = p + j < kv.n_pages && kv.refs[p + j] == 0;
      n += f[j];
    }
    int total;
    int at = found + cta_scan(n, sh, total);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (f[j]) {
        if (at < want) list[at] = p + j;
        ++at;
      }
    found += total;
  }
  return min(found, want);
}

// first[s] = the first list entry that names sequence s; later ones are repeats
__device__ void mark_first(const int32_t* ids, int n, int max_seqs, int* first) {
  for (int i = threadIdx.x; i < max_seqs; i += blockDim.x) first[i] = INT_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int s = ids[i];
    if (s >= 0 && s < max_seqs) atomicMin(&first[s], i);
  }
  __syncthreads();
}

// ---------------------------------------------------------------- reserve
// ws: need[n] (blocks the entry takes), at[n] (their place in the free list), list[n_pages]
__global__ void __launch_bounds__(kPlanThreads)
reserve_kernel(const KvView kv, const int32_t* seqs, const int32_t* n_new, int n, int32_t* need, int32_t* at,
               int32_t* list, uint32_t* status) {
  extern __shared__ int first[];
  __shared__ PlanScan sh;
  __shared__ int s_bad;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) s_bad = 0;
  mark_first(seqs, n, kv.max_seqs, first);
  int total = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int blocks = 0;
    if (i < n) {
      const int s = seqs[i];
      blocks = -1;
      if (s >= 0 && s < kv.max_seqs && n_new[i] >= 0 && first[s] == i) {
        const int len = kv.len_of(s);
        const long long to = (long long)len + n_new[i];
        if (to > ((long long)kv.max_blocks << kv.page_shift) || to > INT_MAX) {
          atomicOr(&s_bad, 1);
          blocks = 0;
        } else {
          blocks = kv.blocks_of((int)to) - kv.blocks_of(len);
        }
      }
      need[i] = blocks;
      if (blocks < 0) set_status(status, MOE_DEV_ERR_BAD_SEQ);
    }
    int sum;
    const int off = cta_scan(max(blocks, 0), sh, sum);
    if (i < n) at[i] = total + off;
    total += sum;   // at most max_seqs * max_blocks, which fits
  }
  const bool full = s_bad != 0 || lowest_free(kv, total, list, sh) < total;   // s_bad: uniform after the scans' barriers
  if (full) {
    if (threadIdx.x == 0) set_status(status, MOE_DEV_ERR_CAPACITY);
    return;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n; i += kPlanThreads / 32) {
    const int blocks = need[i];
    if (blocks < 0) continue;
    const int s = seqs[i], len = kv.len_of(s);
    const int b0 = kv.blocks_of(len);
    for (int b = lane; b < blocks; b += 32) {
      const int p = list[at[i] + b];
      kv.table[(size_t)s * kv.max_blocks + b0 + b] = p;
      kv.refs[p] = 1;
    }
    __syncwarp();
    if (lane == 0) kv.lens[s] = len + n_new[i];
  }
}

// ---------------------------------------------------------------- append
// A warp takes `per` <= 32 rows at a time: one run of bytes to read, `per` places to write (61 MB of rows: 18 us, 6.7
// TB/s read and written; with a thread per 16 bytes that finds its own place 24 us).
__global__ void __launch_bounds__(kApplyThreads)
append_kernel(const KvView kv, int layer, const uint4* rows, const int32_t* tok_seq, const int32_t* tok_pos, unsigned N,
              const AppendShape shape, uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int vecs = kv.row >> 3, lane = threadIdx.x & 31;
  const unsigned per = shape.per, step = append_step(shape);
  for (unsigned i0 = append_first(shape, blockIdx.x, threadIdx.x >> 5); i0 < N; i0 += step) {
    // lane j finds where row i0 + j goes (its dependent reads are the warp's only ones)
    const unsigned i = i0 + lane;
    long long to = -1;
    if (lane < (int)per && i < N) {
      const int s = tok_seq[i], pos = tok_pos[i];
      if (s < 0 || s >= kv.max_seqs || pos < 0 || pos >= kv.len_of(s)) {
        set_status(status, MOE_DEV_ERR_BAD_SEQ);
      } else {
        const int p = kv.table[(size_t)s * kv.max_blocks + (pos >> kv.page_shift)];
        if (p < 0 || p >= kv.n_pages || kv.refs[p] != 1) set_status(status, MOE_DEV_ERR_BAD_PAGE);
        else to = (long long)kv.row_offset(layer, p, pos & (kv.page_tokens - 1));
      }
    }
    const uint4* from = rows + (size_t)i0 * vecs;
    const int total = (int)min(per, N - i0) * vecs;
    for (int x0 = 0; x0 < total; x0 += 32 * 8) {          // eight reads in flight
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int x = x0 + 32 * j + lane;
        if (x < total) v[j] = __ldcs(from + x);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int x = x0 + 32 * j + lane, r = min(x / vecs, 31);
        const long long at = __shfl_sync(0xffffffffu, to, r);
        if (x < total && at >= 0) reinterpret_cast<uint4*>(kv.pages + at)[x - r * vecs] = v[j];
      }
    }
  }
}

// ---------------------------------------------------------------- fork
struct ForkPlan {
  int len;      // the source's length; -1: nothing to do for this pair
  int page;     // the new page of a partly filled last block, or -1
  int from;     // the page it is copied from
  int old_len;  // what the destination held
};

// One CTA: which pairs are valid, which need a page, and which page.  first: one int per sequence in shared memory.
__device__ void fork_plan(const KvView& kv, const int32_t* src, const int32_t* dst, int n, ForkPlan* plan,
                          int32_t* list, int* first, PlanScan& sh, uint32_t* status) {
  mark_first(dst, n, kv.max_seqs, first);
  int total = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    bool part = false;
    ForkPlan f = {-1, -1, -1, 0};
    if (i < n) {
      const int s = src[i], d = dst[i];
      const bool good = s >= 0 && s < kv.max_seqs && d >= 0 && d < kv.max_seqs && first[d] == i;
      if (!good) set_status(status, MOE_DEV_ERR_BAD_SEQ);
      if (good && s != d) {
        f.len = kv.len_of(s);
        f.old_len = kv.len_of(d);
        part = (f.len & (kv.page_tokens - 1)) != 0;
        if (part) f.from = kv.table[(size_t)s * kv.max_blocks + (f.len >> kv.page_shift)];
      }
    }
    int sum;
    const int off = cta_scan(part ? 1 : 0, sh, sum);
    if (part) f.page = total + off;   // its place in the free list, for now
    if (i < n) plan[i] = f;
    total += sum;
  }
  const bool full = lowest_free(kv, total, list, sh) < total;
  if (full && threadIdx.x == 0) set_status(status, MOE_DEV_ERR_CAPACITY);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    ForkPlan f = plan[i];
    if (full) f.len = -1;
    else if (f.page >= 0) f.page = list[f.page];
    plan[i] = f;
  }
}

// The sources' block tables as they were (a source may be another pair's destination): pairs from, from + step, ...
__device__ void fork_snapshot(const KvView& kv, const int32_t* src, const int32_t* dst, int n, int32_t* snap, int from,
                              int step) {
  for (int i = from; i < n; i += step) {
    const int s = src[i];
    if (s < 0 || s >= kv.max_seqs || s == dst[i]) continue;
    const int blocks = kv.blocks_of(kv.len_of(s));
    for (int b = threadIdx.x; b < blocks; b += blockDim.x)
      snap[(size_t)i * kv.max_blocks + b] = kv.table[(size_t)s * kv.max_blocks + b];
  }
}

// One pair's block table and reference counts (the CTA's threads).
__device__ void fork_table(const KvView& kv, int d, const ForkPlan& f, const int32_t* snap) {
  const int blocks = kv.blocks_of(f.len), old_blocks = kv.blocks_of(f.old_len);
  int32_t* row = kv.table + (size_t)d * kv.max_blocks;
  for (int b = threadIdx.x; b < max(blocks, old_blocks); b += blockDim.x) {
    const int was = row[b];
    const int now = b >= blocks ? -1 : (f.page >= 0 && b == blocks - 1) ? f.page : snap[b];
    if (was == now) continue;
    if (was >= 0 && was < kv.n_pages) atomicSub(&kv.refs[was], 1);
    if (now >= 0 && now < kv.n_pages) atomicAdd(&kv.refs[now], 1);
    row[b] = now;
  }
  if (threadIdx.x == 0) kv.lens[d] = f.len;
}

// The valid rows of one pair's partly filled page, every layer: thread `x` of `threads`.
__device__ void fork_copy(const KvView& kv, const ForkPlan& f, int x, int threads, uint32_t* status) {
  if (f.page < 0) return;
  if (f.from < 0 || f.from >= kv.n_pages) {
    if (x == 0) set_status(status, MOE_DEV_ERR_BAD_PAGE);
    return;
  }
  const int vecs = (f.len & (kv.page_tokens - 1)) * (kv.row >> 3);   // the valid rows are one run of bytes
  for (int layer = 0; layer < kv.n_layers; ++layer) {
    const uint4* from = reinterpret_cast<const uint4*>(kv.pages + kv.row_offset(layer, f.from, 0));
    uint4* to = reinterpret_cast<uint4*>(kv.pages + kv.row_offset(layer, f.page, 0));
#pragma unroll 4
    for (int v = x; v < vecs; v += threads) to[v] = from[v];
  }
}

// Two launches, for copies that need the whole GPU: CTA 0 plans while the others take the snapshot, then a row of
// CTAs a pair applies it (block row 0: the table; the others: a share of the page's rows).
__global__ void __launch_bounds__(kPlanThreads)
fork_plan_kernel(const KvView kv, const int32_t* src, const int32_t* dst, int n, ForkPlan* plan, int32_t* list,
                 int32_t* snap, uint32_t* status) {
  extern __shared__ int first[];
  __shared__ PlanScan sh;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) fork_plan(kv, src, dst, n, plan, list, first, sh, status);
  else fork_snapshot(kv, src, dst, n, snap, blockIdx.x - 1, gridDim.x - 1);
}

__global__ void __launch_bounds__(kApplyThreads)
fork_apply_kernel(const KvView kv, const int32_t* dst, const ForkPlan* plan, const int32_t* snap, uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const ForkPlan f = plan[i];
  if (f.len < 0) return;
  if (blockIdx.y == 0) fork_table(kv, dst[i], f, snap + (size_t)i * kv.max_blocks);
  else fork_copy(kv, f, (blockIdx.y - 1) * blockDim.x + threadIdx.x, (gridDim.y - 1) * blockDim.x, status);
}

// One launch of one cluster, for small copies: its CTAs meet between the plan and its application.
__global__ void __launch_bounds__(kPlanThreads) __cluster_dims__(kCluster, 1, 1)
fork_small_kernel(const KvView kv, const int32_t* src, const int32_t* dst, int n, ForkPlan* plan, int32_t* list,
                  int32_t* snap, uint32_t* status) {
  extern __shared__ int first[];
  __shared__ PlanScan sh;
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x;
  if (c == 0) fork_plan(kv, src, dst, n, plan, list, first, sh, status);
  else fork_snapshot(kv, src, dst, n, snap, c - 1, kCluster - 1);
  cluster_meet();
  for (int i = c; i < n; i += kCluster) {
    const ForkPlan f = plan[i];
    if (f.len < 0) continue;
    fork_table(kv, dst[i], f, snap + (size_t)i * kv.max_blocks);
    fork_copy(kv, f, threadIdx.x, kPlanThreads, status);
  }
}

// ---------------------------------------------------------------- free
__global__ void __launch_bounds__(kApplyThreads)
free_kernel(const KvView kv, const int32_t* seqs, uint32_t* status) {
  __shared__ int s_len;
  pdl_wait();
  pdl_trigger();
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= kv.max_seqs) {
    if (threadIdx.x == 0) set_status(status, MOE_DEV_ERR_BAD_SEQ);
    return;
  }
  if (threadIdx.x == 0) {   // whoever takes the length releases the blocks: a repeat finds 0
    const long long cap = (long long)kv.max_blocks << kv.page_shift;
    const int n = atomicExch(&kv.lens[s], 0);
    s_len = n < 0 ? 0 : n > cap ? (int)cap : n;
  }
  __syncthreads();
  int32_t* row = kv.table + (size_t)s * kv.max_blocks;
  for (int b = threadIdx.x; b < kv.blocks_of(s_len); b += blockDim.x) {
    const int p = row[b];
    if (p >= 0 && p < kv.n_pages) atomicSub(&kv.refs[p], 1);
    row[b] = -1;
  }
}

// ---------------------------------------------------------------- compact
// counts[0] = pages that move, counts[1] = n_live; move[j] = (from, to); to[p] = new place of a page that moves
// One CTA.
__device__ void compact_plan(const KvView& kv, int32_t* counts, int32_t* from, int32_t* dest, int32_t* to,
                             int32_t* n_live_opt, PlanScan& sh) {
  int live = 0;
  for (int p = threadIdx.x; p < kv.n_pages; p += kPlanThreads) live += kv.refs[p] != 0;
  int n_live;
  cta_scan(live, sh, n_live);
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < kv.n_pages; p0 += 4 * kPlanThreads) {
    const int p = p0 + 4 * threadIdx.x;
    int kind[4], nh = 0, nm = 0;   // 1: a hole below n_live, 2: a page that moves
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      kind[j] = 0;
      if (p + j < kv.n_pages) {
        const bool used = kv.refs[p + j] != 0;
        kind[j] = !used && p + j < n_live ? 1 : used && p + j >= n_live ? 2 : 0;
      }
      nh += kind[j] == 1;
      nm += kind[j] == 2;
    }
    int th, tm;
    int ah = holes + cta_scan(nh, sh, th), am = movers + cta_scan(nm, sh, tm);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kind[j] == 1) dest[ah++] = p + j;
      if (kind[j] == 2) from[am++] = p + j;
    }
    holes += th;
    movers += tm;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < movers; j += kPlanThreads) {   // as many holes below n_live as pages in use above it
    const int a = from[j], b = dest[j];
    to[a] = b;
    kv.refs[b] = kv.refs[a];
    kv.refs[a] = 0;
  }
  if (threadIdx.x == 0) {
    counts[0] = movers;
    counts[1] = n_live;
    if (n_live_opt) *n_live_opt = n_live;
  }
}

// CTA c of `ctas`: its share of the block tables, and of the pages that move (a page of one layer at a time).
__device__ void compact_apply(const KvView& kv, const int32_t* counts, const int32_t* from, const int32_t* dest,
                              const int32_t* to, int c, int ctas) {
  const int moves = counts[0], n_live = counts[1];
  if (moves == 0) return;
  for (long long e = (long long)c * blockDim.x + threadIdx.x; e < (long long)kv.max_seqs * kv.max_blocks;
       e += (long long)ctas * blockDim.x) {
    const int p = kv.table[e];
    if (p >= n_live && p < kv.n_pages) kv.table[e] = to[p];
  }
  const int vecs = kv.page_tokens * (kv.row >> 3);
  const long long units = (long long)moves * kv.n_layers;
  for (long long u = c; u < units; u += ctas) {
    const int j = (int)(u / kv.n_layers), layer = (int)(u - (long long)j * kv.n_layers);
    const uint4* a = reinterpret_cast<const uint4*>(kv.pages + kv.row_offset(layer, from[j], 0));
    uint4* b = reinterpret_cast<uint4*>(kv.pages + kv.row_offset(layer, dest[j], 0));
#pragma unroll 4
    for (int v = threadIdx.x; v < vecs; v += blockDim.x) b[v] = a[v];
  }
}

__global__ void __launch_bounds__(kPlanThreads)
compact_plan_kernel(const KvView kv, int32_t* counts, int32_t* from, int32_t* dest, int32_t* to, int32_t* n_live_opt) {
  __shared__ PlanScan sh;
  pdl_wait();
  pdl_trigger();
  compact_plan(kv, counts, from, dest, to, n_live_opt, sh);
}

__global__ void __launch_bounds__(kApplyThreads)
compact_apply_kernel(const KvView kv, const int32_t* counts, const int32_t* from, const int32_t* dest,
                     const int32_t* to) {
  pdl_wait();
  pdl_trigger();
  compact_apply(kv, counts, from, dest, to, blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kPlanThreads) __cluster_dims__(kCluster, 1, 1)
compact_small_kernel(const KvView kv, int32_t* counts, int32_t* from, int32_t* dest, int32_t* to, int32_t* n_live_opt) {
  __shared__ PlanScan sh;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) compact_plan(kv, counts, from, dest, to, n_live_opt, sh);
  cluster_meet();
  // as compact_apply, with the pages' bytes as one run of work: four reads in flight a thread
  const int moves = counts[0], n_live = counts[1], tid = blockIdx.x * kPlanThreads + threadIdx.x;
  constexpr int kAll = kCluster * kPlanThreads;
  if (moves == 0) return;
  const int vecs = kv.page_tokens * (kv.row >> 3), total = moves * kv.n_layers * vecs;   // kSmallPool keeps this an int
  for (int x0 = tid; x0 < total; x0 += 4 * kAll) {
    uint4 v[4];
    uint4* at[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int x = x0 + q * kAll;
      if (x < total) {
        const int u = x / vecs, y = x - u * vecs, j = u / kv.n_layers, layer = u - j * kv.n_layers;
        v[q] = reinterpret_cast<const uint4*>(kv.pages + kv.row_offset(layer, from[j], 0))[y];
        at[q] = reinterpret_cast<uint4*>(kv.pages + kv.row_offset(layer, dest[j], 0)) + y;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (x0 + q * kAll < total) *at[q] = v[q];
  }
  for (long long e = tid; e < (long long)kv.max_seqs * kv.max_blocks; e += kAll) {
    const int p = kv.table[e];
    if (p >= n_live && p < kv.n_pages) kv.table[e] = to[p];
  }
}

// Up to these bytes a call runs as one cluster on 8 SMs, from there on as a plan and a launch of the whole GPU.
// Copies of a fork (with a free, us, cluster / two launches): 0.29 MB 9.1 / 9.9, 0.44 MB 10.8 / 9.6, 1.2 MB 18.9 / 9.0.
constexpr long long kSmallCopy = 384ll << 10;
// The pool of a compaction, which the host knows, unlike what moves: with an eighth of the pages free 8 MB 6.8 / 10.6,
// 16 MB 12.5 / 10.1; with half of them free 4 MB 8.2 / 10.5, 8 MB 18.4 / 9.4.
constexpr long long kSmallPool = 8ll << 20;

size_t ints(size_t n) { return align_up(n * sizeof(int32_t), 256); }

size_t kv_ws_bytes(const moe_kv_cache& c, int n) {
  const size_t reserve = 2 * ints(n) + ints(c.n_pages);
  const size_t fork = align_up((size_t)n * sizeof(ForkPlan), 256) + ints(n) + ints((size_t)n * c.max_blocks);
  const size_t compact = ints(2) + 3 * ints(c.n_pages);
  return reserve > fork ? (reserve > compact ? reserve : compact) : (fork > compact ? fork : compact);
}

int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int check_list(const moe_kv_cache* c, const void* a, const void* b, int n) {
  const int st = check_kv(c);
  if (st != MOE_OK) return st;
  if (n < 0 || n > c->max_seqs) return MOE_ERR_INVALID_ARG;
  return n > 0 && (!a || !b) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_kv_workspace_size(const moe_kv_cache* cache, int n) {
  return check_kv(cache) != MOE_OK || n < 0 ? 0 : kv_ws_bytes(*cache, n);
}

int moe_kv_reserve(const moe_kv_cache* cache, const int32_t* seqs, const int32_t* n_new, int n, void* ws,
                   size_t ws_bytes, uint32_t* dev_status, moe_stream_t stream) {
  int st = check_list(cache, seqs, n_new, n);
  if (st != MOE_OK || n == 0) return st;
  st = check_ws(ws, ws_bytes, kv_ws_bytes(*cache, n));
  if (st != MOE_OK) return st;
  char* b = reinterpret_cast<char*>(ws);
  return status_of(launch_k(reserve_kernel, 1, kPlanThreads, (size_t)cache->max_seqs * sizeof(int),
                            reinterpret_cast<cudaStream_t>(stream), kv_view(*cache), seqs, n_new, n,
                            reinterpret_cast<int32_t*>(b), reinterpret_cast<int32_t*>(b + ints(n)),
                            reinterpret_cast<int32_t*>(b + 2 * ints(n)), dev_status));
}

int moe_kv_append(const moe_kv_cache* cache, int layer, const void* rows, const int32_t* tok_seq,
                  const int32_t* tok_pos, int N, uint32_t* dev_status, moe_stream_t stream) {
  const int st = check_kv(cache);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= cache->n_layers || N < 0) return MOE_ERR_INVALID_ARG;
  if (N == 0) return MOE_OK;
  if (!rows || !tok_seq || !tok_pos) return MOE_ERR_INVALID_ARG;
  if (!kv_aligned(rows, 16)) return MOE_ERR_UNSUPPORTED;
  static_assert(kAppendWarps == kApplyThreads / 32, "warps of a CTA");
  const AppendShape shape = append_shape((unsigned)N, (unsigned)num_sms());
  return status_of(launch_k(append_kernel, shape.ctas, kApplyThreads, 0, reinterpret_cast<cudaStream_t>(stream),
                            kv_view(*cache), layer, reinterpret_cast<const uint4*>(rows), tok_seq, tok_pos, (unsigned)N,
                            shape, dev_status));
}

int moe_kv_fork(const moe_kv_cache* cache, const int32_t* src, const int32_t* dst, int n, void* ws,
                size_t ws_bytes, uint32_t* dev_status, moe_stream_t stream) {
  int st = check_list(cache, src, dst, n);
  if (st != MOE_OK || n == 0) return st;
  st = check_ws(ws, ws_bytes, kv_ws_bytes(*cache, n));
  if (st != MOE_OK) return st;
  char* b = reinterpret_cast<char*>(ws);
  ForkPlan* plan = reinterpret_cast<ForkPlan*>(b);
  b += align_up((size_t)n * sizeof(ForkPlan), 256);
  int32_t* list = reinterpret_cast<int32_t*>(b);
  int32_t* snap = reinterpret_cast<int32_t*>(b + ints(n));
  const KvView kv = kv_view(*cache);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t first = (size_t)cache->max_seqs * sizeof(int);
  const long long page_vecs = (long long)cache->n_layers * cache->page_tokens * ((cache->rank + cache->rope) / 8);
  if (n * page_vecs * 16 <= kSmallCopy)
    return status_of(launch_k(fork_small_kernel, kCluster, kPlanThreads, first, s, kv, src, dst, n, plan, list, snap,
                              dev_status));
  cudaError_t e = launch_k(fork_plan_kernel, 1 + (n < 256 ? n : 256), kPlanThreads, first, s, kv, src, dst, n, plan, list,
                           snap, dev_status);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  // copy CTAs of a pair: about 8 16-byte vectors a thread for a full page in every layer
  const long long want = (page_vecs + 8 * kApplyThreads - 1) / (8 * kApplyThreads);
  return status_of(launch_k(fork_apply_kernel, dim3(n, 1 + (unsigned)(want < 64 ? want : 64)), kApplyThreads, 0, s, kv,
                            dst, plan, snap, dev_status));
}

int moe_kv_free(const moe_kv_cache* cache, const int32_t* seqs, int n, uint32_t* dev_status, moe_stream_t stream) {
  const int st = check_list(cache, seqs, seqs, n);
  if (st != MOE_OK || n == 0) return st;
  return status_of(launch_k(free_kernel, n, kApplyThreads, 0, reinterpret_cast<cudaStream_t>(stream), kv_view(*cache),
                            seqs, dev_status));
}

int moe_kv_compact(const moe_kv_cache* cache, int32_t* n_live_opt, void* ws, size_t ws_bytes, uint32_t* dev_status,
                   moe_stream_t stream) {
  int st = check_kv(cache);
  if (st != MOE_OK) return st;
  st = check_ws(ws, ws_bytes, kv_ws_bytes(*cache, 0));
  if (st != MOE_OK) return st;
  (void)dev_status;
  const size_t list = ints(cache->n_pages);
  char* b = reinterpret_cast<char*>(ws);
  int32_t* counts = reinterpret_cast<int32_t*>(b);
  int32_t* from = reinterpret_cast<int32_t*>(b + ints(2));
  int32_t* dest = reinterpret_cast<int32_t*>(b + ints(2) + list);
  int32_t* to = reinterpret_cast<int32_t*>(b + ints(2) + 2 * list);
  const KvView kv = kv_view(*cache);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const long long pool = (long long)cache->n_layers * cache->n_pages * cache->page_tokens * (cache->rank + cache->rope) * 2;
  if (pool <= kSmallPool)
    return status_of(launch_k(compact_small_kernel, kCluster, kPlanThreads, 0, s, kv, counts, from, dest, to, n_live_opt));
  cudaError_t e = launch_k(compact_plan_kernel, 1, kPlanThreads, 0, s, kv, counts, from, dest, to, n_live_opt);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  return status_of(launch_k(compact_apply_kernel, 8 * num_sms(), kApplyThreads, 0, s, kv, counts, from, dest, to));
}

}  // extern "C"
