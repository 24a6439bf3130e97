// Absorbed latent attention over the paged cache: every head's keys are the
// cached rows themselves and its values their first `rank` entries, so all
// heads of a sequence share one pass over its rows.
//
// Per 64-token tile and up to 64 query rows (a row = one query token of one head):
//   S   = Q K^T    M = query rows (64), N = tokens, K = rank + rope
//   O^T += V^T P^T  M = latent entries (128 a slice), N = query rows, K = tokens
// S is taken with the query rows as M so that a row's softmax is one thread's;
// O is taken transposed because 64 rows x 512 entries then fill 4 slices x N
// columns of tensor memory (256 of 512), leaving room for two S tiles, and
// because few heads cost few columns.  V^T reads the very tile K was read
// from: the same shared-memory bytes as an operand with M contiguous.
// P (bf16) overwrites the tile's rotary chunk, which S no longer needs.
//
// Softmax: running maximum m and sum l per row in the log2 domain, fp32.  O is
// rescaled only when a row's maximum rises by more than 2^8: until then the
// old maximum keeps all terms below 2^8 and the sums exact to fp32 as before.
//
// Work: the sequences' tiles form one line that is cut evenly over the CTAs
// (teams of G CTAs where a sequence has G > 1 row tiles, so that its rows are
// read from HBM once and from L2 by the others).  A cut sequence leaves fp32
// partial (O, m, l) per piece; a combine kernel joins the pieces in order.  A
// shared prefix is a second line: row tiles over the whole batch's query rows
// against the prefix's tiles.
//
// Bound: a tile with its 64 rows moves 322 KB through shared memory (Q and K for
// S, V and P for O, the copies in), 2515 cycles at 128 bytes a cycle; its products
// alone take 2230.  Long documents take 4100 a tile, starts, pieces and the join
// included (84 tiles an SM at 2070 MHz).  With fewer heads the rows of the
// cache bound it, and for short sequences the chain launch, lengths, table, copy,
// S, softmax, O, combine.  Measured, rank 512 and rope 64:
//   1 x 333 tokens, 32 heads              12.9 us
//   32 x 250..6001, 64 heads              36.7 us 3.1 TB/s of cached rows
//   4 x 40001..65537, 128 heads, 2 tokens 169 us  0.69 PFLOP/s
//   64 x 16384 shared + 17..1500, 32 heads 127 us 0.60 PFLOP/s
//
// A cache in 4 bits (kv_fp4.cuh) differs in how a tile comes: its codes are staged by
// TMA as they are, and eight more warps expand them into the places that copies of bf16
// rows would fill, a ring of 128-entry pairs.  Products, softmax and pieces are the same,
// and so are the answers, bit for bit those of a bf16 cache of the same values.  It
// holds 2.8 times the tokens; it is not faster: a tile of 64 tokens takes 5100 cycles
// where bf16 takes 3700.  The softmax is the reason (3000 cycles of it where it takes 1100
// alone): its code and the expansion's take turns in the instruction caches, and every copy of the
// expansion that unrolling added made it worse (kv_fp4.cuh).  A prefix that many row tiles read is
// expanded once, to bf16.  Measured, rank 512 and rope 64, with what bf16 takes:
//   1 x 333 tokens, 32 heads              15.2 us  13.2
//   32 x 250..6001, 16 heads              42 us    33.2
//   4 x 40001..65537, 32 heads, 2 tokens  90 us    74
//   64 x 16384 shared + 17..1500, 32 heads 154 us  126
//
// Roles (224 threads): warp 0 = TMA producer, warp 1 = issuer of S (and TMEM
// owner), warps 2..5 = softmax, rescaling and epilogue, warp 6 = issuer of the
// value products (an issuer of its own: a tile's value product frees the tile's
// memory, and must not wait behind the next tile's S, which waits for its loads);
// in 4 bits warps 7..14 expand, warp 15 copies codes.
// Every mbarrier wait is bounded; on expiry the CTA reports
// MOE_DEV_ERR_TIMEOUT, drains and returns.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "kv_fp4.cuh"
#include "latent_line.h"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kChunk = kTok * kBK * 2;   // 8 KB: 64 tokens x 64 entries (also 64 query rows x 64 entries)
constexpr int kMaxPairs = 4;             // 128-entry slices of the latent
constexpr int kMaxSlots = 4;             // tiles in flight
constexpr int kBatch = 512;              // sequences of one launch (lengths and tile sums in shared memory)
constexpr int kThreads = 224;            // a bf16 cache's; one in 4 bits has kExpandWarps more
constexpr int kExpandWarps = 8;          // and one that copies their codes
constexpr int kBufs = 8;                 // pairs of a cache in 4 bits that are expanded at once, at most
constexpr int kStages = 2;               // tiles of rotary keys in flight there (of codes one: its readers hold the one before)
constexpr int kSoftThreads = 128;
constexpr int kTmemCols = 512;
constexpr int kSCol = 256;               // S tiles at columns 256 and 320; O slices at 0, 64, 128, 192
constexpr float kGrow = 8.0f;            // log2 of the growth of a row's maximum that forces a rescaling

struct DecodeParams : LineShape {
  KvView kv;
  int layer, rope;
  int pairs, slots, bufs;    // rank / 128; tiles in flight; in 4 bits, pairs that are expanded at once
  int q_bytes;               // in 4 bits: room of a tile's queries
  int lines;                 // which lines this launch takes: 1 the prefix, 2 the sequences', 3 both
  const int32_t* prefix_blocks;   // the prefix's block table where it is not its sequence's, else nullptr
  float scale_log2;          // scale * log2(e): the exponentials are powers of two
  const int32_t* seqs;
  const int32_t* prefix_seq;
  __nv_bfloat16* out;
  float* lse;
  int32_t* plan;             // [B + 1] tile sums, for the combine
  float* part_s;             // suffix pieces: [2 teams G (+ B G with a prefix)][NR][rank]
  float4* ml_s;              // their (m, l, l of the rounded probabilities)
  float* part_p;             // prefix pieces: [2 ctas + Gp][NRp][rank]
  float4* ml_p;
  uint32_t* status;
};

struct Seg {
  int row0, rows, N;   // query rows
  int b, seq;          // sequence of the batch (suffix) whose tokens these are; its id in the cache
  int tok0, tok1;
  float* part;         // where a piece goes; nullptr: the whole sequence, straight to out
  float4* ml;
  bool prefix;
};

// A CTA's pieces: first of the prefix line, then of the sequences' line, which
// the CTAs take from the other end (calls too small for both lines to fill the
// grid keep them on different SMs).  A sequence stands in its line with kHead
// units ahead of its tiles, for what starting and ending a piece costs.
struct SegIter {
  const DecodeParams& p;
  const int* pref;
  const int* len;
  const int* ids;
  long long pos, end;
  int b, cta, team, g, per;
  bool first;
  int phase;

  __device__ SegIter(const DecodeParams& p_, const int* pref_, const int* len_, const int* ids_)
      : p(p_), pref(pref_), len(len_), ids(ids_) {
    phase = 0;
    const long long total = (long long)p.Gp * p.np;
    pos = min(total, (long long)blockIdx.x * p.per_p);
    end = p.lines & 1 ? min(total, pos + p.per_p) : pos;
    first = true;
  }
  __device__ void start_suffix() {
    phase = 1;
    first = true;
    cta = p.ctas - 1 - blockIdx.x;
    team = cta / p.G;
    g = cta - team * p.G;
    const int total = pref[p.B];
    per = per_cta(total, p.teams);
    pos = team < p.teams ? min((long long)total, (long long)team * per) : total;
    end = min((long long)total, pos + per);
    int lo = 0, hi = p.B;   // the last b with pref[b] <= pos
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pref[mid] <= pos) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  __device__ bool next(Seg& s) {
    const int rank = p.kv.rank;
    if (phase == 0) {
      if (pos < end) {
        const int i = (int)(pos / p.np), x0 = (int)(pos - (long long)i * p.np);
        const int x1 = (int)min((long long)p.np, x0 + end - pos);
        s.prefix = true;
        s.b = 0;
        s.seq = *p.prefix_seq;
        s.row0 = i * p.NRp;
        s.rows = min(p.NRp, p.B * p.Q * p.heads - s.row0);
        s.tok0 = x0 * kTok;
        s.tok1 = min(x1 * kTok, p.shared);
        const int slot = (x0 == 0 && x1 == p.np) ? 2 * p.ctas + i : 2 * blockIdx.x + (first ? 0 : 1);
        s.part = p.part_p + (size_t)slot * p.NRp * rank;
        s.ml = p.ml_p + (size_t)slot * p.NRp;
        s.N = up16(s.rows);
        pos += x1 - x0;
        first = false;
        return true;
      }
      if (!(p.lines & 2)) return false;
      start_suffix();
    }
    if (pos >= end) return false;
    while (pref[b + 1] <= pos) ++b;
    const int n = pref[b + 1] - pref[b] - kHead;
    int x0 = (int)(pos - pref[b]);
    const int x1 = (int)min((long long)n, x0 + end - pos - kHead);
    if (x1 <= 0) return false;             // the range ends within the head of this sequence
    pos = pref[b] + x1 + kHead;
    x0 = max(0, x0 - kHead);
    s.prefix = false;
    s.b = b;
    s.seq = ids[b];
    s.row0 = b * p.Q * p.heads + g * p.NR;
    s.rows = min(p.NR, p.Q * p.heads - g * p.NR);
    s.tok0 = p.shared + x0 * kTok;
    s.tok1 = min(p.shared + x1 * kTok, len[b]);
    const bool whole = x0 == 0 && x1 == n;
    s.part = nullptr;
    s.ml = nullptr;
    if (!whole || p.np) {
      const int slot = whole ? 2 * p.teams * p.G + b * p.G + g : 2 * cta + (first ? 0 : 1);
      s.part = p.part_s + (size_t)slot * p.NR * rank;
      s.ml = p.ml_s + (size_t)slot * p.NR;
    }
    s.N = up16(s.rows);
    first = false;
    return true;
  }
};

// 16 lanes x 64 fp32 columns over a warp: thread t gets, for each group i of 8
// columns, {row t/4, columns 8i + 2(t%4) + 0, 1} and the same of row t/4 + 8.
__device__ inline void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// One thread's latent entry of `rows` accumulator columns (query rows) to dst[row * stride]: 32 lanes write 32
// neighbouring entries of a row at once.
template <typename T>
__device__ inline void store_columns(uint32_t taddr, int rows, int stride, T* dst, const float* factor = nullptr) {
  uint32_t v[2][16];
  tmem_ld16(taddr, v[0]);
#pragma unroll
  for (int c = 0; c < kRows; c += 16) {
    if (c >= rows) break;
    tmem_ld_wait();
    if (c + 16 < rows) tmem_ld16(taddr + c + 16, v[(c >> 4) + 1 & 1]);   // the next block arrives behind these stores
    const int n = rows - c;
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      if (x < n) {
        const float a = __uint_as_float(v[(c >> 4) & 1][x]);
        if constexpr (sizeof(T) == 4) dst[x * stride] = a;
        else dst[x * stride] = __float2bfloat16_rn(a * factor[c + x]);
      }
    }
    dst += 16 * stride;
  }
}

// Two bf16 values, those that are NaN or infinite as 0.
__device__ inline uint32_t finite_bf16x2(uint32_t v) {
  if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
  if ((v & 0x7F800000u) == 0x7F800000u) v &= 0x0000FFFFu;
  return v;
}

__device__ inline float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// OR of a predicate over the softmax warps (named barrier 1): the same answer in every thread.
__device__ inline bool soft_any(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(kSoftThreads)
      : "memory");
  return r != 0;
}

// Four 8 x 8 matrices of 16-bit entries in one store; lane l gives the address of row l % 8 of matrix l / 8.  (One
// store for four: shared memory is busy with the products' operands, and a store waits its turn each time.)
__device__ inline void store_matrices(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

struct alignas(16) Shared {   // its size is what the dynamic shared memory leaves free
  // bf16: per 128-entry pair of a slot, then the rotary chunk.  In 4 bits, one behind the other: a ring of expanded pairs
  // (kBufs), the rotary chunks (kStages), the stage of codes.
  uint64_t full[kMaxSlots][kMaxPairs + 1], empty[kMaxSlots][kMaxPairs + 1];
  uint64_t q_full, q_empty, s_full[2], s_empty[2], p_full[kPBars], pv_done[2], drain[2];
  uint32_t tmem;
  int abort;
  float factor[kRows];   // rescaling of each row; in the epilogue 1 / l
  int warp_sum[kThreads / 32 + kExpandWarps + 1];
  int sees[kSoftThreads / 32];
  unsigned long long bad[2];   // tokens of a tile (by its parity) with a NaN or infinite latent entry, bit by bit
  int pref[kBatch + 1];
  int len[kBatch];
  int ids[kBatch];
};

template <bool FP4>
constexpr int kAllThreads = kThreads + (FP4 ? 32 * (kExpandWarps + 1) : 0);

template <bool FP4>
__global__ void __launch_bounds__(kAllThreads<FP4>, 1)
decode_kernel(const __grid_constant__ CUtensorMap map_kv, const __grid_constant__ CUtensorMap map_pair,
              const __grid_constant__ CUtensorMap map_qs, const __grid_constant__ CUtensorMap map_qsr,
              const __grid_constant__ CUtensorMap map_qp, const __grid_constant__ CUtensorMap map_qpr,
              const __grid_constant__ CUtensorMap map_scales, const DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kAll = kAllThreads<FP4>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunks = 2 * p.pairs + 1;               // the last one holds the rotary part, then P
  uint8_t* skv = smem + (FP4 ? p.q_bytes : chunks * kChunk);
  const int slot_bytes = chunks * kChunk, kv_at = FP4 ? p.q_bytes : slot_bytes;
  // in 4 bits: queries, expanded pairs, rotary chunks, the stage of codes, and their barriers.  The queries' last chunk is
  // read 64 rows deep; the places past its rows are the first pair's.
  uint8_t* srope = skv + (FP4 ? p.bufs * 2 * kChunk : 0);
  uint8_t* sstage = srope + kStages * kChunk;
  uint64_t *const full4 = &sh.full[0][0], *const empty4 = &sh.empty[0][0];
  constexpr int kRopeBar = kBufs, kStageBar = kBufs + kStages;
  static_assert(kStageBar < kMaxSlots * (kMaxPairs + 1), "barriers");
  // A tile comes and goes in these parts: the value product lets go of one pair after the other, and the next tile's
  // copies follow at once (two parts a tile instead of five measured 13% to 20% slower on long sequences).
  const int parts = p.pairs + (p.rope ? 1 : 0);

  if (tid == 0) {
    if (FP4) {
      for (int i = 0; i <= kStageBar; ++i) {
        mbar_init(full4 + i, i < kRopeBar ? kExpandWarps : 1);
        mbar_init(empty4 + i, i < kStageBar ? 1 : kExpandWarps);
      }
    } else {
      for (int s = 0; s < p.slots; ++s)
        for (int j = 0; j <= p.pairs; ++j) {
          mbar_init(&sh.full[s][j], 1);
          mbar_init(&sh.empty[s][j], 1);
        }
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], kSoftThreads / 32);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.drain[i], 1);
    }
    for (int i = 0; i < kPBars; ++i) mbar_init(&sh.p_full[i], 1);
    sh.abort = 0;
    sh.bad[0] = sh.bad[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 32 * 2) {
    prefetch_map(&map_kv);
    prefetch_map(&map_pair);
    if (FP4) prefetch_map(&map_scales);
    prefetch_map(&map_qs);
    prefetch_map(&map_qsr);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();   // the combine's CTAs need no shared memory to speak of: they wait beside these
  // lengths and tile sums of the batch (every CTA for itself)
  {
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAll) {
      const int b = b0 + tid;
      int n = 0;
      if (b < p.B) {
        const int s = p.seqs[b];
        const bool good = s >= 0 && s < p.kv.max_seqs;
        const int len = good ? p.kv.len_of(s) : 0;
        if (!good && blockIdx.x == 0) set_status(p.status, MOE_DEV_ERR_BAD_SEQ);
        sh.len[b] = len;
        sh.ids[b] = s;
        n = len > p.shared ? (len - p.shared + kTok - 1) / kTok + kHead : 0;
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
  SegIter it(p, sh.pref, sh.len, sh.ids);
  Seg sg;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    // The whole warp runs the loop on warp-uniform values; one elected lane issues.
    int tile = 0, nseg = 0, slot = 0;
    uint32_t par = 1;
    bool ok = true;
    const int page = p.kv.page_tokens, box = min(page, kTok);
    const int layer_page = p.layer * p.kv.n_pages, cq = 2 * p.pairs + (p.rope ? 1 : 0);
    const bool pseq_ok = p.np == 0 || (*p.prefix_seq >= 0 && *p.prefix_seq < p.kv.max_seqs);
    const uint32_t smem0 = uni(smem_u32(smem)), kv0 = smem0 + chunks * kChunk;
    const uint32_t full0 = uni(smem_u32(&sh.full[0][0])), qbar = uni(smem_u32(&sh.q_full));
    // rows that only this CTA reads leave L2 to the pieces; rows that others read too stay
    const uint64_t once = l2_evict_first(), shared = l2_normal();
    while (__any_sync(0xffffffffu, ok && it.next(sg))) {
      const bool seq_ok = !sg.prefix || pseq_ok;      // a bad id in the batch has no tokens
      const uint64_t pol = sg.prefix || p.G > 1 ? shared : once;
      const int32_t* blocks = sg.prefix && p.prefix_blocks ? p.prefix_blocks
                                                             : p.kv.table + (seq_ok ? (size_t)sg.seq * p.kv.max_blocks : 0);
      const int tok0 = (int)uni(sg.tok0), tok1 = (int)uni(sg.tok1);
      // lane i: the pool row where box i of a tile begins; read one tile ahead
      auto block = [&](int t) { return seq_ok && lane < kTok / box && t < tok1 ? blocks[t >> p.kv.page_shift] : -1; };
      int ahead = block(tok0 + lane * box);
      const int row0 = (int)uni(sg.row0);
      // the queries follow the first tile: the tile's memory is free before the last piece's S lets go of its queries
      auto load_q = [&]() {
        if (!warp_wait(&sh.q_empty, (nseg & 1) ^ 1u, abort_flag)) return false;
        // the tile's rows, chunk behind chunk of box rows (rows past the tile's are read and not used)
        const CUtensorMap* mq = sg.prefix ? &map_qp : &map_qs;
        const CUtensorMap* mr = sg.prefix ? &map_qpr : &map_qsr;
        const int q_rows = sg.prefix ? p.NRp : p.NR;
        mbar_expect_tx_warp(qbar, (uint32_t)(cq * q_rows * 128));
        ++nseg;
        tma_load_3d_hint_warp(smem0, mq, qbar, 0, row0, 0, shared);
        if (p.rope) tma_load_2d_warp(smem0 + 2 * p.pairs * q_rows * 128, mr, qbar, p.kv.rank, row0);
        return true;
      };
      const bool q_first = nseg == 0;
      if (q_first) ok = load_q();
      for (int t0 = tok0; ok && t0 < tok1; t0 += kTok) {
        const int nb = (min(kTok, tok1 - t0) + box - 1) / box;       // boxes that hold tokens
        const int t = t0 + lane * box;
        int row = ahead;
        if (lane < nb) {
          if (row < 0 || row >= p.kv.n_pages) {
            set_status(p.status, seq_ok ? MOE_DEV_ERR_BAD_PAGE : MOE_DEV_ERR_BAD_SEQ);
            row = 0;
          }
          row = (layer_page + row) * page + (t & (page - 1));
        } else {
          row = 0;
        }
        ahead = block(t + kTok);
        int rows[kTok / 16];
#pragma unroll
        for (int i = 0; i < kTok / 16; ++i) rows[i] = (int)uni(lane == i ? row : 0);
        if (FP4) {                   // the rotary keys alone
          if (p.rope) {
            ok = warp_wait(empty4 + kRopeBar + slot, par, abort_flag);
            if (ok) {
              const uint32_t to = uni(smem_u32(srope)) + slot * kChunk, fb = full0 + 8 * (kRopeBar + slot);
              mbar_expect_tx_warp(fb, (uint32_t)(nb * box * 128));
#pragma unroll
              for (int i = 0; i < kTok / 16; ++i)
                if (i < nb) tma_load_2d_hint_warp(to + i * box * 128, &map_kv, fb, p.kv.rope_at, rows[i], pol);
            }
          }
        } else {
          const uint32_t dst = kv0 + slot * slot_bytes, bar = full0 + slot * (uint32_t)sizeof(sh.full[0]);
          for (int j = 0; j < parts; ++j) {
            ok = warp_wait(&sh.empty[slot][j], par, abort_flag);
            if (!ok) break;
            const bool pair = j < p.pairs;
            const uint32_t to = dst + 2 * j * kChunk, fb = bar + 8 * j;
            mbar_expect_tx_warp(fb, (uint32_t)(nb * box * (pair ? 256 : 128)));
            if (box == kTok && pair) {   // both chunks of the pair in one copy
              tma_load_3d_hint_warp(to, &map_pair, fb, 0, rows[0], 2 * j, pol);
            } else {
#pragma unroll
              for (int i = 0; i < kTok / 16; ++i)
                if (i < nb) {
                  tma_load_2d_hint_warp(to + i * box * 128, &map_kv, fb, 2 * j * kBK, rows[i], pol);
                  if (pair) tma_load_2d_hint_warp(to + kChunk + i * box * 128, &map_kv, fb, 2 * j * kBK + kBK, rows[i], pol);
                }
            }
          }
        }
        if (ok && t0 == tok0 && !q_first) ok = load_q();
        ++tile;
        if (++slot == p.slots) {
          slot = 0;
          par ^= 1u;
        }
      }
    }
    // drain: whatever was asked for lands before the CTA can exit (a barrier's
    // latest load is its latest phase; after an abort the last tile's barriers
    // may not all be armed, and the bounded wait outlasts any copy)
    volatile int no_abort = 0;
    if (nseg) mbar_wait(&sh.q_full, (nseg - 1) & 1, &no_abort);
    for (int s = 0; s < p.slots; ++s) {
      const int loads = tile / p.slots + (tile % p.slots > s ? 1 : 0);
      if (FP4) {
        if (loads > 0 && p.rope) mbar_wait(full4 + kRopeBar + s, (loads - 1) & 1, &no_abort);
      } else {
        for (int j = 0; j < parts; ++j)
          if (loads > 0) mbar_wait(&sh.full[s][j], (loads - 1) & 1, &no_abort);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ issuer of S
    // The whole warp runs the loop on warp-uniform values; one elected lane issues.
    int tile = 0, nseg = 0, slot = 0;
    uint32_t par = 0;
    bool issued = false, ok = true;
    constexpr uint32_t idesc_s = make_idesc(64, kTok);
    const uint32_t tm = uni(tmem), smem0 = uni(smem_u32(smem));
    const uint64_t dq0 = smem_desc(smem0), dk0 = smem_desc(smem0 + kv_at), dr0 = smem_desc(uni(smem_u32(srope)));
    int buf4 = 0;
    uint32_t par4 = 0;
    while (__any_sync(0xffffffffu, ok && it.next(sg))) {
      ok = warp_wait(&sh.q_full, nseg & 1, abort_flag);
      const int n_tiles = (int)uni((sg.tok1 - sg.tok0 + kTok - 1) / kTok);
      const uint64_t q_step = (uint64_t)((uni(sg.prefix ? p.NRp : p.NR) * 128) >> 4);   // from one chunk of the queries to the next
      for (int i = 0; ok && i < n_tiles; ++i, ++tile) {
        const int buf = tile & 1;
        ok = warp_wait(&sh.s_empty[buf], ((tile >> 1) & 1) ^ 1u, abort_flag);
        if (!ok) break;
        uint64_t dq = dq0, dk = dk0 + ((uint64_t)(slot * slot_bytes) >> 4);
        const uint32_t d = tm + kSCol + buf * kTok;
        for (int j = 0; j < p.pairs; ++j) {
          ok = warp_wait(FP4 ? full4 + buf4 : &sh.full[slot][j], FP4 ? par4 : par, abort_flag);
          if (!ok) break;
          if (FP4) {
            dk = dk0 + ((uint64_t)(buf4 * 2 * kChunk) >> 4);
            if (++buf4 == p.bufs) {
              buf4 = 0;
              par4 ^= 1u;
            }
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_warp(d, dq + ((k & 3) * kUK * 2 >> 4) + (k >> 2) * q_step,
                        dk + (((k >> 2) * kChunk + (k & 3) * kUK * 2) >> 4), idesc_s, k ? 1u : (j ? 1u : 0u));
          issued = true;
          dq += 2 * q_step;
          dk += (2 * kChunk) >> 4;
        }
        if (ok && p.rope) {
          ok = warp_wait(FP4 ? full4 + kRopeBar + slot : &sh.full[slot][p.pairs], par, abort_flag);
          if (ok) {
            if (FP4) dk = dr0 + ((uint64_t)(slot * kChunk) >> 4);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k * kUK < p.rope) tc_mma_warp(d, dq + ((k * kUK * 2) >> 4), dk + ((k * kUK * 2) >> 4), idesc_s, 1u);
          }
        }
        if (!ok) break;
        tc_commit_warp(&sh.s_full[buf]);
        if (i == n_tiles - 1) tc_commit_warp(&sh.q_empty);
        if (++slot == p.slots) {
          slot = 0;
          par ^= 1u;
        }
      }
      ++nseg;
    }
    if (issued) {   // every issued product completes before tensor memory is released
      volatile int no_abort = 0;
      tc_commit_warp(&sh.drain[0]);
      mbar_wait(&sh.drain[0], 0, &no_abort);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------------ issuer of the value products
    int tile = 0, slot = 0;
    bool issued = false, ok = true;
    const uint32_t tm = uni(tmem), smem0 = uni(smem_u32(smem));
    const uint64_t dv0 = smem_desc_mn(smem0 + kv_at, kChunk);
    const uint64_t dp0 = FP4 ? smem_desc(uni(smem_u32(srope))) : smem_desc(smem0 + kv_at) + (uint64_t)((2 * p.pairs * kChunk) >> 4);
    int buf4 = 0;
    while (__any_sync(0xffffffffu, ok && it.next(sg))) {
      const int n_tiles = (int)uni((sg.tok1 - sg.tok0 + kTok - 1) / kTok);
      const uint32_t idesc = make_idesc(128, (int)uni(sg.N)) | kTransA;
      for (int i = 0; i < n_tiles; ++i, ++tile) {
        ok = warp_wait(&sh.p_full[p_bar(tile)], p_phase(tile), abort_flag);   // P is written, so S has read the whole tile
        if (!ok) break;
        tc_fence_after();
        const uint64_t step = (uint64_t)(slot * (FP4 ? kChunk : slot_bytes)) >> 4;
        uint64_t dv = dv0 + step;
        const uint64_t dp = dp0 + step;
        for (int j = 0; j < p.pairs; ++j) {
          if (FP4) dv = dv0 + ((uint64_t)(buf4 * 2 * kChunk) >> 4);
#pragma unroll
          for (int k = 0; k < kTok / kUK; ++k)
            tc_mma_warp(tm + j * kRows, dv + ((k * kUK * 128) >> 4), dp + ((k * kUK * 2) >> 4), idesc,
                        k ? 1u : (i ? 1u : 0u));
          tc_commit_warp(FP4 ? empty4 + buf4 : &sh.empty[slot][j]);
          dv += (2 * kChunk) >> 4;
          if (FP4 && ++buf4 == p.bufs) buf4 = 0;
        }
        if (p.rope) tc_commit_warp(FP4 ? empty4 + kRopeBar + slot : &sh.empty[slot][p.pairs]);
        tc_commit_warp(&sh.pv_done[tile & 1]);
        issued = true;
        if (++slot == p.slots) slot = 0;
      }
    }
    if (issued) {
      volatile int no_abort = 0;
      tc_commit_warp(&sh.drain[1]);
      mbar_wait(&sh.drain[1], 0, &no_abort);
    }
    __syncwarp();
  } else if (FP4 && warp == kThreads / 32 + kExpandWarps) {
    // ------------------------------------------------ copies of codes and scales, as they are
    int tile = 0;
    bool ok = true;
    const int page = p.kv.page_tokens, box = min(page, kTok), layer_page = p.layer * p.kv.n_pages;
    const int regions = fp4_regions(p.kv.rank);
    const uint32_t to = uni(smem_u32(sstage)), bar = uni(smem_u32(full4 + kStageBar));
    const bool pseq_ok = p.np == 0 || (*p.prefix_seq >= 0 && *p.prefix_seq < p.kv.max_seqs);
    const uint64_t once = l2_evict_first(), shared = l2_normal();
    while (__any_sync(0xffffffffu, ok && it.next(sg))) {
      const bool seq_ok = !sg.prefix || pseq_ok;
      const uint64_t pol = sg.prefix || p.G > 1 ? shared : once;
      const int32_t* blocks = sg.prefix && p.prefix_blocks ? p.prefix_blocks
                                                             : p.kv.table + (seq_ok ? (size_t)sg.seq * p.kv.max_blocks : 0);
      const int tok0 = (int)uni(sg.tok0), tok1 = (int)uni(sg.tok1);
      auto block = [&](int t) { return seq_ok && lane < kTok / box && t < tok1 ? blocks[t >> p.kv.page_shift] : -1; };
      int ahead = block(tok0 + lane * box);
      for (int t0 = tok0; ok && t0 < tok1; t0 += kTok) {
        const int nb = (min(kTok, tok1 - t0) + box - 1) / box;       // boxes that hold tokens
        const int t = t0 + lane * box;
        int row = ahead;
        if (lane < nb) {
          if (row < 0 || row >= p.kv.n_pages) {
            set_status(p.status, seq_ok ? MOE_DEV_ERR_BAD_PAGE : MOE_DEV_ERR_BAD_SEQ);
            row = 0;
          }
          row = (layer_page + row) * page + (t & (page - 1));
        } else {
          row = 0;
        }
        ahead = block(t + kTok);
        ok = warp_wait(empty4 + kStageBar, (tile & 1) ^ 1u, abort_flag);
        if (!ok) break;
        mbar_expect_tx_warp(bar, (uint32_t)(nb * box * (128 * regions + 32)));
#pragma unroll 1
        for (int i = 0; i < nb; ++i) {
          const int r = (int)uni(__shfl_sync(0xffffffffu, row, i));
#pragma unroll 1
          for (int g = 0; g < regions; ++g)
            tma_load_2d_hint_warp(to + g * kTok * 128 + i * box * 128, &map_pair, bar, 128 * g, r, pol);
          tma_load_2d_hint_warp(to + regions * kTok * 128 + i * box * 32, &map_scales, bar, p.kv.rank / 2 + 2 * p.rope, r, pol);
        }
        ++tile;
      }
    }
    volatile int no_abort = 0;
    if (tile) mbar_wait(full4 + kStageBar, (tile - 1) & 1, &no_abort);
    __syncwarp();
  } else if (FP4 && warp >= kThreads / 32) {
    // ------------------------------------------------ latents in 4 bits, expanded into the pairs that a copy would fill
    // Four threads a token; of each 128-entry pair a thread has 16 bytes of codes, a quarter.  A tile's codes go to
    // registers at once, so that the next tile's are on their way while these are expanded.  Places past a piece's last
    // token get whatever the stage holds, which the softmax warps hide and clear.
    const int r = (warp - kThreads / 32) * 8 + (lane & 7), v = lane >> 3;
    const int regions = fp4_regions(p.kv.rank);
    const Fp4Place to(smem_u32(skv), kChunk, r, v);
    const uint32_t stage = smem_u32(sstage);
    int buf = 0, tile = 0;
    uint32_t par = 1;
    bool ok = true;
    while (__any_sync(0xffffffffu, ok && it.next(sg))) {
      const int n_tiles = (sg.tok1 - sg.tok0 + kTok - 1) / kTok;
      for (int i = 0; ok && i < n_tiles; ++i, ++tile) {
        ok = warp_wait(full4 + kStageBar, tile & 1, abort_flag);
        if (!ok) break;
        uint4 c[kMaxPairs];
        uint32_t scales[kMaxPairs];
#pragma unroll
        for (int j = 0; j < kMaxPairs; ++j)
          if (j < p.pairs) fp4_fetch(stage, kTok, regions, r, v, j, c[j], scales[j]);
        __syncwarp();
        if (lane == 0) mbar_arrive(empty4 + kStageBar);
#pragma unroll 1
        for (int j = 0; j < p.pairs; ++j) {
          ok = warp_wait(empty4 + buf, par, abort_flag);
          if (!ok) break;
          fp4_store32<1>(to, buf * 2 * kChunk, c[0], scales[0]);
          proxy_fence();
          __syncwarp();
          if (lane == 0) mbar_arrive(full4 + buf);
          if (++buf == p.bufs) {
            buf = 0;
            par ^= 1u;
          }
#pragma unroll
          for (int x = 0; x + 1 < kMaxPairs; ++x) {       // rolled: one copy of the expansion
            c[x] = c[x + 1];
            scales[x] = scales[x + 1];
          }
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax, rescaling, epilogue
    // S has 64 rows, 16 lanes of tensor memory in each warp's quarter.  A thread
    // holds rows r and r + 8 of its warp's 16 and columns 8 i + 2 (lane % 4) + {0, 1}
    // of both: four threads share a row, and all 32 lanes have work.
    const int quarter = warp & 3, st = tid - 64, c2 = 2 * (lane & 3);
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const int r0 = quarter * 16 + (lane >> 2);
    const int rank = p.kv.rank;
    int tile = 0;
    bool fail = false;
    const float scale = p.scale_log2;
    const float unseen = scale >= 0.0f ? -INFINITY : INFINITY;   // what a token out of sight scores
    // Where this lane's matrix row goes in P: row lane % 8 of the warp's 16 (+ 8: 1024 bytes on), 16-byte column group
    // lane / 8 (+ 4: bit 6 flips), swizzled with the row.
    const uint32_t p_row = (quarter * 16 + (lane & 7)) * 128, p_at0 = ((lane >> 3) ^ (lane & 7)) << 4;
    if (st < kRows) sh.factor[st] = 1.0f;
    while (!fail && it.next(sg)) {
      int limit[2];
      bool active[2];
      float m[2];
      float2 l[2];   // sums of the probabilities, and of what they are rounded to (this thread's columns)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + 8 * e;
        active[e] = r < sg.rows;
        limit[e] = 0;
        if (active[e]) {
          const int bq = (sg.row0 + r) / p.heads, b = bq / p.Q;
          limit[e] = sh.len[b] - p.Q + (bq - b * p.Q) + 1;
        }
        m[e] = -INFINITY;
        l[e] = make_float2(0.0f, 0.0f);
      }
      // tokens up to here are seen by all of the warp's rows, and by all of the tile's
      int sees_all = __reduce_min_sync(0xffffffffu, min(active[0] ? limit[0] : INT_MAX, active[1] ? limit[1] : INT_MAX));
      if (lane == 0) sh.sees[quarter] = sees_all;
      soft_any(false);                      // and the factors are set
      const int sees_tile = min(min(sh.sees[0], sh.sees[1]), min(sh.sees[2], sh.sees[3]));
      sees_all = min(sees_all, sg.tok1);
      for (int t0 = sg.tok0; t0 < sg.tok1; t0 += kTok, ++tile) {
        const int buf = tile & 1, slot = tile % p.slots;
        // where the tile's pair j lies
        auto pair_at = [&](int j) { return skv + (FP4 ? (tile * p.pairs + j) % p.bufs * 2 * kChunk : slot * slot_bytes + 2 * j * kChunk); };
        const int n_tok = min(kTok, sg.tok1 - t0);
        // The product of two tiles ago is long over; waiting for each in turn keeps its barrier's phase unambiguous.
        const bool ok = (tile < 2 || warp_wait(&sh.pv_done[buf], ((tile - 2) >> 1) & 1, abort_flag)) &&
                        warp_wait(&sh.s_full[buf], (tile >> 1) & 1, abort_flag);
        float s[32];   // [i][e][2]
        if (ok) {
          tc_fence_after();
          tmem_ld_rows16(lane_base + kSCol + buf * kTok, reinterpret_cast<uint32_t(&)[32]>(s));
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.s_empty[buf]);
        }
        bool grow = !ok;
        float ref[2];
        if (t0 + kTok > sees_all) {
          // some row does not see all 64 tokens
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int see = min(n_tok, limit[e] - t0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (8 * i + c2 >= see) s[4 * i + 2 * e] = unseen;
              if (8 * i + c2 + 1 >= see) s[4 * i + 2 * e + 1] = unseen;
            }
          }
        }
        if (t0 + n_tok > sees_tile) {
          // Some row does not see some token (the last tile of several query tokens): its probability 0 times a NaN or
          // infinite value would be NaN.  Such values become 0 here, and a row that does see the token gets NaN through
          // its score: the value may have made that -infinity, whose product with the value is NaN as well.
          unsigned long long bad = 0;
          if (ok) {
            for (int j = 0; j < p.pairs; ++j) {
              if (FP4) mbar_wait(full4 + (tile * p.pairs + j) % p.bufs, (tile * p.pairs + j) / p.bufs & 1, abort_flag);
              else mbar_wait(&sh.full[slot][j], (tile / p.slots) & 1, abort_flag);   // long over
              uint4* base = reinterpret_cast<uint4*>(pair_at(j));
              for (int x = st; x < 2 * kChunk / 16; x += kSoftThreads) {
                const uint4 v = base[x];
                const uint4 f = make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z), finite_bf16x2(v.w));
                if (((v.x ^ f.x) | (v.y ^ f.y) | (v.z ^ f.z) | (v.w ^ f.w)) != 0) {
                  base[x] = f;
                  bad |= 1ull << ((x & (kChunk / 16 - 1)) >> 3);   // a token's row is 128 bytes of a chunk
                }
              }
            }
            if (bad) atomicOr(&sh.bad[buf], bad);
          }
          if (soft_any(bad != 0)) {
            bad = sh.bad[buf];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int see = min(n_tok, limit[e] - t0);
#pragma unroll
              for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  if (8 * i + c2 + y < see && (bad >> (8 * i + c2 + y) & 1)) s[4 * i + 2 * e + y] = NAN;
            }
          }
        }
        float top[2];
        if (scale >= 0.0f) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float a = fmaxf(s[2 * e], s[2 * e + 1]), b = fmaxf(s[4 + 2 * e], s[5 + 2 * e]);
#pragma unroll
            for (int i = 2; i < 8; i += 2) {
              a = fmaxf(fmaxf(a, s[4 * i + 2 * e]), s[4 * i + 2 * e + 1]);
              b = fmaxf(fmaxf(b, s[4 * i + 4 + 2 * e]), s[4 * i + 5 + 2 * e]);
            }
            top[e] = fmaxf(a, b);
          }
#pragma unroll
          for (int o = 1; o <= 2; o <<= 1)
#pragma unroll
            for (int e = 0; e < 2; ++e) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[e] = s[2 * e];
#pragma unroll
            for (int i = 0; i < 8; ++i) top[e] = fminf(top[e], fminf(s[4 * i + 2 * e], s[4 * i + 2 * e + 1]));
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) top[e] = fminf(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float now = limit[e] > t0 ? top[e] * scale : -INFINITY;
          if (active[e] && now > m[e] + (m[e] == -INFINITY ? 0.0f : kGrow)) {
            if (m[e] != -INFINITY) {        // else nothing is summed for this row yet
              const float f = ex2(m[e] - now);
              l[e].x *= f;
              l[e].y *= f;
              grow = true;
              if ((lane & 3) == 0) sh.factor[r0 + 8 * e] = f;
            }
            m[e] = now;
          }
          ref[e] = m[e] == -INFINITY ? 0.0f : m[e];
        }
        // Probabilities, rounded to bf16 (the cache's type, the only one the product takes beside it).  Their sum is of
        // the rounded ones: the output is divided by it, so its weights add up to one, and where few tokens carry the
        // row most of their rounding cancels.  The log-sum-exp wants the sum of the unrounded ones too.
        const uint32_t sp = smem_u32(FP4 ? srope + slot * kChunk : skv + slot * slot_bytes + 2 * p.pairs * kChunk) + p_row;
        auto probabilities = [&](auto with_lse) {
          if (quarter * 16 >= sg.N) return;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 mul = make_float2(scale, scale), sub = make_float2(-ref[e], -ref[e]);
            float2 sum = make_float2(0.0f, 0.0f), rsum = sum;
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 x = fma2(make_float2(s[4 * i + 2 * e], s[4 * i + 2 * e + 1]), mul, sub);
              x.x = ex2(x.x);
              x.y = ex2(x.y);
              const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
              w[i] = *reinterpret_cast<const uint32_t*>(&h);
              if (decltype(with_lse)::value) sum = add2(sum, x);
              rsum = add2(rsum, make_float2(bf16_lo(w[i]), bf16_hi(w[i])));
            }
            store_matrices(sp + e * 1024 + p_at0, w[0], w[1], w[2], w[3]);
            store_matrices(sp + e * 1024 + (p_at0 ^ 64), w[4], w[5], w[6], w[7]);
            l[e].x += sum.x + sum.y;
            l[e].y += rsum.x + rsum.y;
          }
        };
        if (p.lse) probabilities(std::true_type{});
        else probabilities(std::false_type{});
        if (n_tok < kTok) {
          // places past the last token: any bits may stand there, and 0 * NaN is NaN
          const int rows = kTok - n_tok;
          for (int j = 0; j < p.pairs; ++j)
            for (int x = st; x < rows * 16; x += kSoftThreads) {
              const int c = x >= rows * 8, y = x - c * rows * 8;
              *reinterpret_cast<uint4*>(pair_at(j) + c * kChunk + n_tok * 128 + y * 16) = make_uint4(0, 0, 0, 0);
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (soft_any(grow)) {      // rare: some row's maximum rose by more than 2^8 (or a wait ran out)
          // O was last added to by the previous tile's product, and this tile's waits for us
          const bool done = ok && warp_wait(&sh.pv_done[buf ^ 1], ((tile - 1) >> 1) & 1, abort_flag);
          fail = soft_any(!done);
          if (fail) break;
          tc_fence_after();
          for (int j = 0; j < p.pairs; ++j)
            for (int c = 0; c < sg.N; c += 16) {
              uint32_t v[16];
              tmem_ld16(lane_base + j * kRows + c, v);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * sh.factor[c + x]);
              tmem_st16(lane_base + j * kRows + c, v);
            }
          tmem_st_wait();
          tc_fence_before();
          soft_any(false);       // everyone has read the factors
          if (st < kRows) sh.factor[st] = 1.0f;
          soft_any(false);
        }
        if (st == 0) {
          sh.bad[buf] = 0;         // read by everyone before the vote above; the next tile writes the other one
          tc_fence_before();
          mbar_arrive(&sh.p_full[p_bar(tile)]);
        }
      }
      if (fail) break;
      const bool done = (tile < 2 || warp_wait(&sh.pv_done[tile & 1], ((tile - 2) >> 1) & 1, abort_flag)) &&
                        warp_wait(&sh.pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1, abort_flag);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
          l[e].x += __shfl_xor_sync(0xffffffffu, l[e].x, o);
          l[e].y += __shfl_xor_sync(0xffffffffu, l[e].y, o);
        }
        const int r = r0 + 8 * e;
        if ((lane & 3) == 0) {
          sh.factor[r] = l[e].y == 0.0f ? 0.0f : 1.0f / l[e].y;
          if (active[e]) {
            if (sg.part) sg.ml[r] = make_float4(m[e], l[e].x, l[e].y, 0.0f);
            else if (p.lse)
              p.lse[sg.row0 + r] = l[e].x == 0.0f ? -INFINITY : (m[e] + log2f(l[e].x)) * 0.6931471805599453f;
          }
        }
      }
      fail = soft_any(!done);
      if (fail) break;
      tc_fence_after();
      const int dim = quarter * 32 + lane;
      if (sg.part) {
        float* dst = sg.part + dim;
        for (int j = 0; j < p.pairs; ++j, dst += 128) store_columns(lane_base + j * kRows, sg.rows, rank, dst);
      } else {
        __nv_bfloat16* dst = p.out + (size_t)sg.row0 * rank + dim;
        for (int j = 0; j < p.pairs; ++j, dst += 128)
          store_columns(lane_base + j * kRows, sg.rows, rank, dst, sh.factor);
      }
      tc_fence_before();
      soft_any(false);
      if (st < kRows) sh.factor[st] = 1.0f;
    }
  }
  __syncthreads();
  if (*abort_flag && tid == 0) set_status(p.status, MOE_DEV_ERR_TIMEOUT);
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// ---------------------------------------------------------------- combine
// Per query row: its pieces' (m, l, O) in a fixed order (the prefix's pieces,
// then the sequence's).  Bound by its dependent reads at small sizes and by L2
// at large ones.
//
// For up to 32 sequences every warp makes them from the lengths while it waits
// for decode_kernel (whose start says that what came before it is complete, so
// the lengths are final; read from L2 all the same): one read less in the chain
// behind it.  Larger batches read the sums that decode_kernel wrote.
constexpr int kEarly = 32;
__device__ inline LineSums early_sums(const DecodeParams& p, int b, int lane) {
  int n = 0;
  if (lane < p.B) {
    const int s = __ldcg(p.seqs + lane);
    int len = s >= 0 && s < p.kv.max_seqs ? __ldcg(p.kv.lens + s) : 0;
    len = (int)min((long long)max(len, 0), (long long)p.kv.max_blocks << p.kv.page_shift);
    n = len > p.shared ? (len - p.shared + kTok - 1) / kTok + kHead : 0;
  }
  int inc = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  LineSums l;
  l.total = __shfl_sync(0xffffffffu, inc, 31);
  l.x1 = __shfl_sync(0xffffffffu, inc, b);
  l.x0 = l.x1 - __shfl_sync(0xffffffffu, n, b);
  return l;
}

// Whether the shared tokens, if any, are a sequence's of the cache.  Where not, no row has a piece: the other rows'
// pieces are made of whatever page stood in for the missing ones.  Asked before the wait, as the lengths.
__device__ inline bool prefix_ok(const DecodeParams& p) {
  return (unsigned)(p.np ? __ldcg(p.prefix_seq) : 0) < (unsigned)p.kv.max_seqs;
}

// Waits for decode_kernel; the whole warp.
__device__ inline LineSums wait_for_pieces(const DecodeParams& p, int row, int lane) {
  const int b = row / (p.Q * p.heads);
  LineSums l;
  if (p.B <= kEarly) l = early_sums(p, b, lane);
  pdl_wait();
  pdl_trigger();
  if (p.B > kEarly) l = LineSums{p.plan[p.B], p.plan[b], p.plan[b + 1]};
  return l;
}

// Piece k of a row, whose place is `at`: its (m, l, l of the rounded probabilities), and its values.
__device__ inline float4 piece_stats(const DecodeParams& p, const Pieces& q, int k, size_t at) {
  return (k < q.n_p ? p.ml_p : p.ml_s)[at];
}
__device__ inline const float4* piece_values(const DecodeParams& p, const Pieces& q, int k, size_t at) {
  return reinterpret_cast<const float4*>((k < q.n_p ? p.part_p : p.part_s) + at * p.kv.rank);
}

// The row's reference maximum and its two sums over all pieces, in every lane.
__device__ inline void join_stats(const DecodeParams& p, const Pieces& q, int lane, float& ref, float& l, float& lr) {
  float top = -INFINITY;
  l = lr = 0.0f;
  size_t at;
  for (int k = lane; q.find(k, at); k += 32) {
    const float4 ml = piece_stats(p, q, k, at);
    const float now = fmaxf(top, ml.x), to = now == -INFINITY ? 0.0f : now;
    const float f = ex2(top - to), w = ex2(ml.x - to);
    l = fmaf(l, f, ml.y * w);
    lr = fmaf(lr, f, ml.z * w);
    top = now;
  }
  const float all = warp_max(top);
  ref = all == -INFINITY ? 0.0f : all;
  const float f = ex2(top - ref);
  l = warp_sum(l * f);
  lr = warp_sum(lr * f);
}

__device__ inline void add_scaled(float4& acc, float w, const float4& x) {
  acc.x = fmaf(w, x.x, acc.x);
  acc.y = fmaf(w, x.y, acc.y);
  acc.z = fmaf(w, x.z, acc.z);
  acc.w = fmaf(w, x.w, acc.w);
}

__device__ inline void store_row(const DecodeParams& p, int row, int v, const float4& acc, float lr) {
  const float inv = lr == 0.0f ? 0.0f : 1.0f / lr;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 packed;
  packed.x = *reinterpret_cast<const uint32_t*>(&lo);
  packed.y = *reinterpret_cast<const uint32_t*>(&hi);
  reinterpret_cast<uint2*>(p.out + (size_t)row * p.kv.rank)[v] = packed;
}

__device__ inline void store_lse(const DecodeParams& p, int row, float ref, float l) {
  if (p.lse) p.lse[row] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
}

// Many rows: a warp a row, up to 4 float4 a lane, four pieces in flight.
__global__ void __launch_bounds__(128) combine_rows_kernel(const DecodeParams p, int rows) {
  const int row = min((int)(blockIdx.x * 4 + (threadIdx.x >> 5)), rows - 1), lane = threadIdx.x & 31;
  const int vecs = p.kv.rank / 128;
  const bool any = prefix_ok(p);
  const LineSums line = wait_for_pieces(p, row, lane);
  Pieces q(p, row, line);
  if (!any) q.n = 0;
  if (q.direct() || blockIdx.x * 4 + (threadIdx.x >> 5) >= rows) return;
  float4 x[4][4];
  float top[4];
  auto load = [&](int k0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      top[j] = -INFINITY;
      size_t at;
      if (q.find(k0 + j, at)) {
        const float4* from = piece_values(p, q, k0 + j, at) + lane;
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (y < vecs) x[j][y] = __ldcs(from + 32 * y);
        top[j] = piece_stats(p, q, k0 + j, at).x;
      }
    }
  };
  load(0);                       // the first values come with the statistics
  float ref, l, lr;
  join_stats(p, q, lane, ref, l, lr);
  float4 acc[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < q.n; k0 += 4) {
    if (k0) load(k0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float w = ex2(top[j] - ref);
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (y < vecs && k0 + j < q.n) add_scaled(acc[y], w, x[j][y]);
    }
  }
#pragma unroll
  for (int y = 0; y < 4; ++y)
    if (y < vecs) store_row(p, row, lane + 32 * y, acc[y], lr);
  if (lane == 0) store_lse(p, row, ref, l);
}

// Few rows, many pieces each: a CTA a row, rank / 128 warps across it and four sets of them over the pieces, which
// meet in shared memory.
constexpr int kSets = 4;
__global__ void __launch_bounds__(128 * kSets) combine_parts_kernel(const DecodeParams p) {
  __shared__ float4 s_acc[128 * kSets];
  const int row = blockIdx.x, lane = threadIdx.x & 31;
  const bool any = prefix_ok(p);
  const LineSums line = wait_for_pieces(p, row, lane);
  Pieces q(p, row, line);
  if (!any) q.n = 0;
  if (q.direct()) return;
  const int v = threadIdx.x % 128, set = threadIdx.x / 128;   // float4 of the row; set of warps
  const bool mine = 4 * v < p.kv.rank;
  float4 x[8];
  float top[8];
  auto load = [&](int k0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = k0 + j * kSets;
      x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      top[j] = -INFINITY;
      size_t at;
      if (mine && q.find(k, at)) {
        x[j] = __ldcs(piece_values(p, q, k, at) + v);
        top[j] = piece_stats(p, q, k, at).x;
      }
    }
  };
  load(set);                     // the first eight values come with the statistics
  float ref, l, lr;
  join_stats(p, q, lane, ref, l, lr);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = set; k0 < q.n; k0 += 8 * kSets) {
    if (k0 != set) load(k0);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k0 + j * kSets < q.n) add_scaled(acc, ex2(top[j] - ref), x[j]);
  }
  s_acc[threadIdx.x] = acc;
  __syncthreads();
  if (set > 0 || !mine) return;
  for (int i = 1; i < kSets; ++i) add_scaled(acc, 1.0f, s_acc[i * 128 + v]);
  store_row(p, row, v, acc, lr);
  if (threadIdx.x == 0) store_lse(p, row, ref, l);
}

// ---------------------------------------------------------------- a prefix in 4 bits, once for all row tiles
// The shared tokens' rows as bf16 pages of the workspace, and those pages' block table.
__global__ void __launch_bounds__(128) unpack_prefix_kernel(const DecodeParams p, __nv_bfloat16* pages, int32_t* table) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31, seq = *p.prefix_seq;
  if (t >= p.shared) return;
  if (lane == 0 && (t & (p.kv.page_tokens - 1)) == 0) table[t >> p.kv.page_shift] = t >> p.kv.page_shift;
  if (seq < 0 || seq >= p.kv.max_seqs) return;                    // reported, and answered with zeros, by those that follow
  int pg = p.kv.table[(size_t)seq * p.kv.max_blocks + (t >> p.kv.page_shift)];
  if (pg < 0 || pg >= p.kv.n_pages) {
    if (lane == 0) set_status(p.status, MOE_DEV_ERR_BAD_PAGE);
    pg = 0;
  }
  const int rank = p.kv.rank, vecs = (rank + p.rope) >> 3;
  const uint8_t* from = reinterpret_cast<const uint8_t*>(p.kv.pages + p.kv.row_offset(p.layer, pg, t & (p.kv.page_tokens - 1)));
  uint4* to = reinterpret_cast<uint4*>(pages) + (size_t)t * vecs;
  const int b = lane, rope_vecs = p.rope >> 3;
  if (b < rank / kFpBlock) {                                      // rank is 512 at most
    const uint2 c = *reinterpret_cast<const uint2*>(from + 8 * b);
    const uint32_t f = fp4_factor(from[rank / 2 + 2 * p.rope + b]);
    to[2 * b] = fp4_expand8(c.x, f);
    to[2 * b + 1] = fp4_expand8(c.y, f);
  }
  if (lane < rope_vecs) to[rank / 8 + lane] = reinterpret_cast<const uint4*>(from + rank / 2)[lane];
}

// ---------------------------------------------------------------- host side
// A prefix in 4 bits that many row tiles read is expanded once, to bf16 pages that they read in its place.  With 32 heads,
// expanded by each / once: 64 sequences over 16384 shared tokens (54 tiles of a row tile a CTA) 184 / 154 us, 16 over 65536
// (54) 177 / 165, 64 over 2048 (7) 67 / 73, 16 over 16384 (13) 76 / 78.
// (Rises with the rows and the shared tokens, as the workspace has to.)
bool unpack_pays(const DecodeParams& p) { return p.np > 0 && p.Gp >= 8 && (long long)p.Gp * p.np >= 24LL * p.ctas; }

struct DecodeWs {
  size_t plan, part_s, ml_s, part_p, ml_p, pages, table, bytes;
};

void fill_shape(DecodeParams& p, const moe_kv_cache& c, int B, int Q, int heads, int shared) {
  set_line(p, B, Q, heads, shared, num_sms());
  p.rope = c.rope;
  p.pairs = c.rank / 128;
}

DecodeWs decode_ws(const DecodeParams& p, const moe_kv_cache& c) {
  const int rank = c.rank;
  DecodeWs w;
  const size_t ns = suffix_rows(p), np = prefix_rows(p);
  w.plan = 0;
  size_t at = align_up((size_t)(p.B + 1) * sizeof(int32_t), 256);
  w.part_s = at;
  at += align_up(ns * rank * sizeof(float), 256);
  w.ml_s = at;
  at += align_up(ns * sizeof(float4), 256);
  w.part_p = at;
  at += align_up(np * rank * sizeof(float), 256);
  w.ml_p = at;
  at += align_up(np * sizeof(float4), 256);
  w.pages = at;              // the prefix as bf16
  w.table = at;
  if (c.format == MOE_KV_FP4 && unpack_pays(p)) {
    w.table += align_up((size_t)p.shared * (rank + c.rope) * 2, 256);
    at = w.table + align_up((size_t)p.shared / 16 * sizeof(int32_t), 256);
  }
  w.bytes = at;
  return w;
}

bool decode_shape_ok(int B, int Q, int heads) { return B <= 4096 && (long long)Q * heads <= 1024; }

template <bool FP4>
cudaError_t launch_decode_kernel(const DecodeParams& p, int smem, cudaStream_t s, const CUtensorMap& kv, const CUtensorMap& pair,
                                 const CUtensorMap& qs, const CUtensorMap& qsr, const CUtensorMap& qp,
                                 const CUtensorMap& qpr, const CUtensorMap& scales) {
  static std::atomic<unsigned char> attr[kMaxDevices];
  const cudaError_t e = once_per_device(attr, [] {
    return cudaFuncSetAttribute(decode_kernel<FP4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                227 * 1024 - (int)sizeof(Shared));
  });
  return e == cudaSuccess
             ? launch_k(decode_kernel<FP4>, p.ctas, kAllThreads<FP4>, smem, s, kv, pair, qs, qsr, qp, qpr, scales, p)
             : e;
}

// One launch of the main kernel over p.kv, whose rows are in 4 bits or not.
cudaError_t launch_lines(DecodeParams p, bool fp4, const void* q, cudaStream_t s) {
  static_assert(sizeof(Shared) + 1024 + (2 * kMaxPairs + 1) * kChunk * 3 <= 227 * 1024, "shared memory");
  static_assert(sizeof(Shared) + 1024 + (2 * kMaxPairs + 1) * kChunk + kStages * kChunk + kTok * (256 + 32) +
                        (kMaxPairs + 1) * 2 * kChunk <= 227 * 1024, "more pairs than a tile has");
  const int rank = p.kv.rank, row = rank + p.rope, slot = (2 * p.pairs + 1) * kChunk;
  int smem;
  if (fp4) {
    // Queries of up to 48 rows leave room for two tiles' pairs; with 64 rows of rank 512 there are 7 of the 8.
    const int q_rows = p.np && p.NRp > p.NR ? p.NRp : p.NR;
    p.q_bytes = ((2 * p.pairs + 1) * q_rows * 128 + 1023) & ~1023;
    const int rest = p.q_bytes + kStages * kChunk + fp4_stage_bytes(rank, kTok) + 1024;
    p.slots = kStages;
    p.bufs = (int)((227 * 1024 - sizeof(Shared) - rest) / (2 * kChunk));
    if (p.bufs > 2 * p.pairs) p.bufs = 2 * p.pairs;
    smem = rest + p.bufs * 2 * kChunk;
  } else {
    p.slots = (int)((227 * 1024 - sizeof(Shared) - 1024 - slot) / slot);   // what the query tile leaves
    if (p.slots > kMaxSlots) p.slots = kMaxSlots;
    smem = (1 + p.slots) * slot + 1024;
  }
  // cache rows by chunk and by pair (in 4 bits: rotary keys, codes and scales); query tiles of sequences and of the prefix
  CUtensorMap kv, pair, qs, qsr, qp, qpr, scales;
  const uint64_t rows = (uint64_t)p.kv.n_layers * p.kv.n_pages * p.kv.page_tokens, qrows = (uint64_t)p.B * p.Q * p.heads;
  const uint32_t box = p.kv.page_tokens < kTok ? p.kv.page_tokens : kTok;
  if (!make_map(&kv, p.kv.pages, p.kv.row, rows, box) || !make_map_chunks(&qs, q, row, qrows, p.NR, 2 * p.pairs) ||
      !make_map(&qsr, q, row, qrows, p.NR))
    return cudaErrorInvalidValue;
  if (fp4 ? !make_map_bytes(&pair, p.kv.pages, 2 * p.kv.row, rows, 128, box, true) ||
                !make_map_bytes(&scales, p.kv.pages, 2 * p.kv.row, rows, 32, box, false)
          : !make_map_chunks(&pair, p.kv.pages, row, rows, kTok, 2))
    return cudaErrorInvalidValue;
  if (!fp4) scales = kv;
  qp = qs;
  qpr = qsr;
  if (p.np && p.NRp != p.NR &&
      (!make_map_chunks(&qp, q, row, qrows, p.NRp, 2 * p.pairs) || !make_map(&qpr, q, row, qrows, p.NRp)))
    return cudaErrorInvalidValue;
  return fp4 ? launch_decode_kernel<true>(p, smem, s, kv, pair, qs, qsr, qp, qpr, scales)
             : launch_decode_kernel<false>(p, smem, s, kv, pair, qs, qsr, qp, qpr, scales);
}

// unpacked: bf16 pages and their block table in the workspace (nullptr: it has no room for them); `there`: an earlier
// launch of the call has filled them
int launch_decode(const moe_kv_cache& c, DecodeParams p, const void* q, __nv_bfloat16* unpacked, int32_t* blocks, bool& there,
                  cudaStream_t s) {
  const bool fp4 = c.format == MOE_KV_FP4;
  cudaError_t e = cudaSuccess;
  p.lines = 3;
  p.prefix_blocks = nullptr;
  if (unpacked && unpack_pays(p)) {
    if (!there) e = launch_k(unpack_prefix_kernel, (unsigned)(p.shared + 3) / 4, 128, 0, s, p, unpacked, blocks);
    there = true;
    DecodeParams first = p;
    first.kv.pages = unpacked;
    first.kv.n_layers = 1;
    first.kv.n_pages = p.shared >> p.kv.page_shift;
    first.kv.row = p.kv.rank + p.rope;
    first.kv.rope_at = p.kv.rank;
    first.layer = 0;
    first.prefix_blocks = blocks;
    first.lines = 1;
    if (e == cudaSuccess) e = launch_lines(first, false, q, s);
    p.lines = 2;
  }
  if (e == cudaSuccess) e = launch_lines(p, fp4, q, s);
  const uint64_t qrows = (uint64_t)p.B * p.Q * p.heads;
  // a CTA a row while the rows alone do not fill the SMs (then a row has many pieces), else a warp a row: whole calls over
  // 1200 tokens a sequence, us, CTA / warp: 128 rows 13.5 / 16.5, 160 rows 16.2 / 16.5, 288 rows 17.6 / 16.5, 1216 rows
  // 37.6 / 24.7
  if (e == cudaSuccess)
    e = qrows <= (uint64_t)p.ctas ? launch_k(combine_parts_kernel, (unsigned)qrows, 128 * kSets, 0, s, p)
                               : launch_k(combine_rows_kernel, (unsigned)((qrows + 3) / 4), 128, 0, s, p, (int)qrows);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_latent_decode_workspace_size(const moe_kv_cache* cache, int B, int Q, int heads, int shared_tokens) {
  if (check_latent(cache, 0) != MOE_OK || B < 1 || Q < 1 || heads < 1 || shared_tokens < 0) return 0;
  if (!decode_shape_ok(B, Q, heads)) return 0;
  DecodeParams p = {};
  fill_shape(p, *cache, B < kBatch ? B : kBatch, Q, heads, shared_tokens);
  return decode_ws(p, *cache).bytes;
}

int moe_latent_decode(const moe_kv_cache* cache, int layer, const void* q, const int32_t* seqs, int B, int Q,
                      int heads, float scale, int shared_tokens, void* out, float* lse_opt, void* ws, size_t ws_bytes,
                      uint32_t* dev_status, moe_stream_t stream) {
  int st = check_latent(cache, layer);
  if (st == MOE_ERR_INVALID_ARG || check_kv(cache) != MOE_OK) return st;
  if (B < 0 || Q < 1 || heads < 1 || shared_tokens < 0 || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (shared_tokens % cache->page_tokens || shared_tokens / cache->page_tokens > cache->max_blocks)
    return MOE_ERR_INVALID_ARG;
  if (B > 0 && (!q || !seqs || !out)) return MOE_ERR_INVALID_ARG;
  if (st != MOE_OK) return st;
  if (!decode_shape_ok(B, Q, heads)) return MOE_ERR_UNSUPPORTED;
  if (B == 0) return MOE_OK;
  if (!kv_aligned(q, 16) || !kv_aligned(out, 16)) return MOE_ERR_UNSUPPORTED;
  st = check_ws(ws, ws_bytes, moe_latent_decode_workspace_size(cache, B, Q, heads, shared_tokens));
  if (st != MOE_OK) return st;
  __nv_bfloat16* pages = nullptr;      // a prefix in 4 bits as bf16: where the first launch's workspace has room for it
  int32_t* blocks = nullptr;
  bool unpacked = false;
  for (int b0 = 0; b0 < B && st == MOE_OK; b0 += kBatch) {   // batches of more than 512 sequences: several launches
    DecodeParams p = {};
    fill_shape(p, *cache, B - b0 < kBatch ? B - b0 : kBatch, Q, heads, shared_tokens);
    const DecodeWs w = decode_ws(p, *cache);
    char* base = reinterpret_cast<char*>(ws);
    const size_t row0 = (size_t)b0 * Q * heads;
    if (b0 == 0 && w.pages < w.table) {      // the first launch's shape, which the workspace is sized by, decides
      pages = reinterpret_cast<__nv_bfloat16*>(base + w.pages);
      blocks = reinterpret_cast<int32_t*>(base + w.table);
    }
    p.kv = kv_view(*cache);
    p.layer = layer;
    // zero as the smallest normal number: a token out of sight scores -infinity, and 0 * -infinity is NaN
    p.scale_log2 = scale == 0.0f ? FLT_MIN : scale * 1.4426950408889634f;
    p.seqs = seqs + b0;
    p.prefix_seq = seqs;
    p.out = reinterpret_cast<__nv_bfloat16*>(out) + row0 * cache->rank;
    p.lse = lse_opt ? lse_opt + row0 : nullptr;
    p.plan = reinterpret_cast<int32_t*>(base + w.plan);
    p.part_s = reinterpret_cast<float*>(base + w.part_s);
    p.ml_s = reinterpret_cast<float4*>(base + w.ml_s);
    p.part_p = reinterpret_cast<float*>(base + w.part_p);
    p.ml_p = reinterpret_cast<float4*>(base + w.ml_p);
    p.status = dev_status;
    st = launch_decode(*cache, p, reinterpret_cast<const __nv_bfloat16*>(q) + row0 * (cache->rank + cache->rope),
                       pages, blocks, unpacked, reinterpret_cast<cudaStream_t>(stream));
  }
  return st;
}

}  // extern "C"
