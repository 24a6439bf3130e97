// Eviction from the latent cache: sequences past a budget keep their heaviest
// tokens.  select_kernel finds, per sequence and layer, which tokens stay; move_kernel
// closes the gaps in place, and the last of a sequence's CTAs shortens its block table.
//
// Selection: the weight that the last token to stay has, found a byte at a time from
// the top (a histogram of those that share the bytes found so far), then a mask and a
// prefix count per 32 tokens.  Of equal weights the first ones stay, by their order in
// the sequence and not by arrival: the same tokens on every run.
// Moves: the order is kept, so every token behind the first gap moves, once, to
// a lower place.  A row is cut into slices that move without knowing of each other.
//
// Bound: rows that move, read and written once (HBM), and for few sequences the
// chains of dependent reads: 8 sequences of 520..700 tokens to 512, one layer: 13 us
// (with a reserve for the next chunk 16.8); 32 of 2500..8192 to 4096, 4 layers, 515 MB: 84
// us, 6.1 TB/s (82 to 91 with the reserve, over 4-bit rows 55).  A sequence is walked by one CTA a slice and chosen from
// by one CTA a layer, however long: half of 16,001 tokens takes 60 us and of 65,537 220, one layer or four, bf16 or 4 bits.
#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveSteps = 4;            // 16-byte loads of a chunk that a thread has in flight

struct EvictPlan {
  int seq;        // -1: nothing to do for this entry
  int len, now;   // tokens before and after
  int head;       // tokens before this all stay
};

struct EvictParams {
  KvView kv;
  int n, budget, first, recent, cap, words;   // cap = max_blocks * page_tokens; words = masks of a sequence and layer
  const int32_t* seqs;
  float* weights;
  int32_t* kept;          // or null
  EvictPlan* plan;        // [n]
  uint32_t* mask;         // [n_layers][n][words] bit t % 32 of word t / 32: token t stays
  int32_t* before;        // [n_layers][n][words] tokens that stay before the word's
  int32_t* done;          // [n] CTAs of move_kernel that have moved their share
  uint32_t* status;
};

// Weights in ascending order as unsigned numbers: a NaN above all, -0 as 0.
__device__ inline uint32_t order_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct SelShared {
  int bad, blocks_shared;
  int hist[256];
  int warp_gt[32], warp_eq[32];
  uint32_t digit;
  int left;
};

constexpr int kHeld = 8;                 // words of 32 weights that a warp keeps in registers: sequences up to 8192 tokens

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictParams p) {
  __shared__ SelShared sh;
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seq = p.seqs[i];
  if (tid == 0) {
    if (layer == 0) p.done[i] = 0;
    sh.bad = 0;
    sh.blocks_shared = 0;
  }
  __syncthreads();
  const bool in_range = seq >= 0 && seq < p.kv.max_seqs;
  if (!in_range) {
    if (tid == 0) sh.bad = MOE_DEV_ERR_BAD_SEQ;
  } else {
    for (int j = tid; j < i; j += kSelThreads)
      if (p.seqs[j] == seq) sh.bad = MOE_DEV_ERR_BAD_SEQ;
  }
  __syncthreads();
  const int len = in_range ? p.kv.len_of(seq) : 0;
  const bool over = sh.bad == 0 && len > p.budget;
  // A warp takes a run of words of 32 tokens, a lane a token of each.  The first words' weights stay in registers; they
  // are on their way while the block table is looked through.
  const int words = (len + 31) / 32, per = (words + 31) / 32, w0 = min(words, warp * per), w1 = min(words, w0 + per);
  const float* w = p.weights + ((size_t)layer * p.kv.max_seqs + (in_range ? seq : 0)) * p.cap;
  float raw[kHeld];
  if (over) {
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
      const int t = (w0 + x) * 32 + lane;
      raw[x] = w0 + x < w1 && t < len ? w[t] : 0.0f;
    }
  }
  if (over) {
    const int32_t* row = p.kv.table + (size_t)seq * p.kv.max_blocks;
    int last = 0;
    bool missing = false;
    for (int b = tid; b < p.kv.blocks_of(len); b += kSelThreads) {
      const int pg = row[b];
      if (pg < 0 || pg >= p.kv.n_pages) missing = true;
      else if (p.kv.refs[pg] > 1) last = b + 1;
    }
    if (missing) atomicOr(&sh.bad, (int)MOE_DEV_ERR_BAD_PAGE);
    if (last) atomicMax(&sh.blocks_shared, last);
  }
  __syncthreads();
  const int bad = sh.bad;
  if (bad) {
    if (tid == 0) {
      set_status(p.status, (uint32_t)bad);
      if (layer == 0) p.plan[i] = EvictPlan{-1, 0, 0, 0};
    }
    return;
  }
  int32_t* kept = p.kept ? p.kept + ((size_t)layer * p.n + i) * p.cap : nullptr;
  if (!over) {
    if (tid == 0 && layer == 0) p.plan[i] = EvictPlan{-1, len, len, len};
    if (kept)
      for (int t = tid; t < len; t += kSelThreads) kept[t] = t;
    return;
  }
  const int head = min(len, max(p.first, sh.blocks_shared << p.kv.page_shift));
  const int tail = max(head, len - p.recent);                  // tokens from here on stay
  const int now = max(p.budget, head + len - tail);
  const int want = now - head - (len - tail);                  // of the tokens between them, fewer than there are
  if (tid == 0 && layer == 0) p.plan[i] = EvictPlan{seq, len, now, head};

  // Key 0: a place that is not chosen among (it lies in the head or the tail, or past the end).
  auto key_of = [&](int word, float weight) {
    const int t = word * 32 + lane;
    return t >= head && t < tail ? order_key(weight) : 0u;   // a weight's own key is above 0 (-infinity: 0x007FFFFF)
  };
  auto key_at = [&](int word) {
    const int t = word * 32 + lane;
    return key_of(word, t < len ? w[t] : 0.0f);
  };
  uint32_t held[kHeld];
#pragma unroll
  for (int x = 0; x < kHeld; ++x) held[x] = w0 + x < w1 ? key_of(w0 + x, raw[x]) : 0u;

  // the want-th largest key, digit by digit; `left` of the keys equal to it stay
  uint32_t prefix = 0;
  int left = want;
  if (want > 0) {
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int d = tid; d < 256; d += kSelThreads) sh.hist[d] = 0;
      __syncthreads();
      // weights of a context crowd into few digits: lanes with one digit add together
      auto count = [&](uint32_t k) {
        const bool in = k != 0 && (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)));
        if (!__any_sync(0xffffffffu, in)) return;
        const uint32_t d = in ? k >> shift & 255 : 256u;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        if (in && lane == __ffs(same) - 1) atomicAdd(&sh.hist[d], __popc(same));
      };
#pragma unroll
      for (int x = 0; x < kHeld; ++x)
        if (w0 + x < w1) count(held[x]);
      for (int x = w0 + kHeld; x < w1; ++x) count(key_at(x));
      __syncthreads();
      if (warp == 0) {             // the digit whose keys, with those above it, first reach `left`
        int mine[8], sum = 0;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          mine[y] = sh.hist[255 - (8 * lane + y)];
          sum += mine[y];
        }
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += u;
        }
        before -= sum;
        if (before < left && before + sum >= left) {
          int l = left - before, y = 0;
#pragma unroll
          for (int z = 0; z < 7; ++z)
            if (y == z && mine[z] < l) {
              l -= mine[z];
              y = z + 1;
            }
          sh.digit = (uint32_t)(255 - (8 * lane + y));
          sh.left = l;
        }
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      left = sh.left;
    }
  }
  // masks: keys above the threshold stay, and the first `left` of those equal to it
  auto classify = [&](int word, uint32_t k, uint32_t& sure, uint32_t& equal) {
    const int t = word * 32 + lane;
    sure = __ballot_sync(0xffffffffu, t < head || (t >= tail && t < len) || (want > 0 && k > prefix));
    equal = __ballot_sync(0xffffffffu, want > 0 && k == prefix);
  };
  int gt = 0, eq = 0;
  auto tally = [&](int word, uint32_t k) {
    uint32_t s, e;
    classify(word, k, s, e);
    gt += __popc(s);
    eq += __popc(e);
  };
#pragma unroll
  for (int x = 0; x < kHeld; ++x)
    if (w0 + x < w1) tally(w0 + x, held[x]);
  for (int x = w0 + kHeld; x < w1; ++x) tally(x, key_at(x));
  if (lane == 0) {
    sh.warp_gt[warp] = gt;
    sh.warp_eq[warp] = eq;
  }
  __syncthreads();
  int at = 0, equals = 0;                 // what stays before this warp's words; keys equal to the threshold before them
  {
    const int g = lane < warp ? sh.warp_gt[lane] : 0, e = lane < warp ? sh.warp_eq[lane] : 0;
    at = __reduce_add_sync(0xffffffffu, g);
    equals = __reduce_add_sync(0xffffffffu, e);
  }
  at += min(equals, left);
  uint32_t* mask = p.mask + ((size_t)layer * p.n + i) * p.words;
  int32_t* before = p.before + ((size_t)layer * p.n + i) * p.words;
  auto mark = [&](int word, uint32_t k) {
    uint32_t s, e;
    classify(word, k, s, e);
    const bool mine = (e >> lane & 1) && equals + __popc(e & ((1u << lane) - 1)) < left;
    const uint32_t m = s | __ballot_sync(0xffffffffu, mine);
    if (lane == 0) {
      mask[word] = m;
      before[word] = at;
    }
    if (kept && (m >> lane & 1)) kept[at + __popc(m & ((1u << lane) - 1))] = word * 32 + lane;
    at += __popc(m);
    equals += __popc(e);
  };
#pragma unroll
  for (int x = 0; x < kHeld; ++x)
    if (w0 + x < w1) mark(w0 + x, held[x]);
  for (int x = w0 + kHeld; x < w1; ++x) mark(x, key_at(x));
}

// The last of a sequence's CTAs (all layers) takes the pages behind the new length out of its block table.
__device__ inline void finish(const EvictParams& p, int i, const EvictPlan& e, int slices) {
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(&p.done[i], 1) == (slices + 1) * p.kv.n_layers - 1;
  }
  __syncthreads();
  if (!s_last) return;
  int32_t* row = p.kv.table + (size_t)e.seq * p.kv.max_blocks;
  for (int b = p.kv.blocks_of(e.now) + threadIdx.x; b < p.kv.blocks_of(e.len); b += kMoveThreads) {
    atomicSub(&p.kv.refs[row[b]], 1);
    row[b] = -1;
  }
  if (threadIdx.x == 0) p.kv.lens[e.seq] = e.now;
}

// In place: a token never moves to a later place, and a chunk of tokens is read before any of it is written, so what a
// chunk writes lies before everything that a later one reads.  A CTA moves VECS 16-byte vectors of every row, the last CTA
// the weights.  Its chunks come one after the other, so that few sequences are narrow slices, long chunks and more CTAs.
template <int VECS>
__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const EvictParams p, int slices) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.y, layer = blockIdx.z, tid = threadIdx.x;
  const EvictPlan e = p.plan[i];
  if (e.seq < 0 || e.now == e.len) return;
  const uint32_t* mask = p.mask + ((size_t)layer * p.n + i) * p.words;
  const int32_t* before = p.before + ((size_t)layer * p.n + i) * p.words;
  const int32_t* table = p.kv.table + (size_t)e.seq * p.kv.max_blocks;
  if ((int)blockIdx.x == slices) {
    float* w = p.weights + ((size_t)layer * p.kv.max_seqs + e.seq) * p.cap;
    for (int t0 = e.head; t0 < e.len; t0 += kMoveThreads * kMoveSteps) {
      float v[kMoveSteps];
#pragma unroll
      for (int u = 0; u < kMoveSteps; ++u) {
        const int t = t0 + u * kMoveThreads + tid;
        if (t < e.len) v[u] = w[t];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kMoveSteps; ++u) {
        const int t = t0 + u * kMoveThreads + tid;
        if (t < e.len) {
          const uint32_t m = mask[t >> 5], bit = 1u << (t & 31);
          if (m & bit) w[before[t >> 5] + __popc(m & (bit - 1))] = v[u];
        }
      }
    }
    __syncthreads();
    for (int t = e.now + tid; t < e.len; t += kMoveThreads) w[t] = 0.0f;
    finish(p, i, e, slices);
    return;
  }
  const int vecs = p.kv.row >> 3, v = blockIdx.x * VECS + (tid % VECS);
  constexpr int kRowsStep = kMoveThreads / VECS, kChunk = kRowsStep * kMoveSteps;
  const bool mine = v < vecs;
  auto place = [&](int t) {
    return reinterpret_cast<uint4*>(p.kv.pages + p.kv.row_offset(layer, table[t >> p.kv.page_shift], t & (p.kv.page_tokens - 1))) + v;
  };
  uint4 x[2][kMoveSteps];
  int to[2][kMoveSteps];
  auto read = [&](int t0, uint4 (&x)[kMoveSteps], int (&to)[kMoveSteps]) {
#pragma unroll
    for (int u = 0; u < kMoveSteps; ++u) {
      const int t = t0 + u * kRowsStep + tid / VECS;
      to[u] = -1;
      if (mine && t < e.len) {
        const uint32_t m = mask[t >> 5], bit = 1u << (t & 31);
        if (m & bit) {
          const int d = before[t >> 5] + __popc(m & (bit - 1));
          if (d != t) {
            to[u] = d;
            x[u] = *place(t);
          }
        }
      }
    }
  };
  auto write = [&](const uint4 (&x)[kMoveSteps], const int (&to)[kMoveSteps]) {
#pragma unroll
    for (int u = 0; u < kMoveSteps; ++u)
      if (to[u] >= 0) *place(to[u]) = x[u];
  };
  // two chunks in turn: a chunk's reads are on their way while the one before is written
  read(e.head, x[0], to[0]);
  for (int t0 = e.head; t0 < e.len; t0 += 2 * kChunk) {
    if (t0 + kChunk < e.len) read(t0 + kChunk, x[1], to[1]);
    __syncthreads();               // everyone has read the first chunk
    write(x[0], to[0]);
    if (t0 + kChunk >= e.len) break;
    if (t0 + 2 * kChunk < e.len) read(t0 + 2 * kChunk, x[0], to[0]);
    __syncthreads();
    write(x[1], to[1]);
  }
  finish(p, i, e, slices);
}

struct EvictWs {
  size_t plan, mask, before, done, bytes;
};

EvictWs evict_ws(const moe_kv_cache& c, int n) {
  const size_t words = ((size_t)c.max_blocks * c.page_tokens + 31) / 32 * n * c.n_layers;
  EvictWs w;
  w.plan = 0;
  w.mask = align_up((size_t)n * sizeof(EvictPlan), 256);
  w.before = w.mask + align_up(words * 4, 256);
  w.done = w.before + align_up(words * 4, 256);
  w.bytes = w.done + align_up((size_t)n * 4, 256);
  return w;
}

bool evict_shape_ok(const moe_kv_cache& c) {
  return (long long)c.max_blocks * c.page_tokens <= (1 << 20) && c.n_layers <= 65535;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_kv_evict_workspace_size(const moe_kv_cache* cache, int n) {
  return check_kv(cache) != MOE_OK || n < 0 || !evict_shape_ok(*cache) ? 0 : evict_ws(*cache, n).bytes;
}

int moe_kv_evict(const moe_kv_cache* cache, const int32_t* seqs, int n, float* weights, int budget, int first,
                 int recent, int32_t* kept_opt, void* ws, size_t ws_bytes, uint32_t* dev_status,
                 moe_stream_t stream) {
  int st = check_kv(cache);
  if (st != MOE_OK) return st;
  if (n < 0 || n > cache->max_seqs || budget < 1 || first < 0 || recent < 0 || (long long)first + recent > budget)
    return MOE_ERR_INVALID_ARG;
  if (n > 0 && (!seqs || !weights)) return MOE_ERR_INVALID_ARG;
  if (!evict_shape_ok(*cache)) return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!kv_aligned(weights, 4) || !kv_aligned(kept_opt, 4)) return MOE_ERR_UNSUPPORTED;
  const EvictWs w = evict_ws(*cache, n);
  st = check_ws(ws, ws_bytes, w.bytes);
  if (st != MOE_OK) return st;
  char* b = reinterpret_cast<char*>(ws);
  EvictParams p;
  p.kv = kv_view(*cache);
  p.n = n;
  p.budget = budget;
  p.first = first;
  p.recent = recent;
  p.cap = cache->max_blocks * cache->page_tokens;
  p.words = (p.cap + 31) / 32;
  p.seqs = seqs;
  p.weights = weights;
  p.kept = kept_opt;
  p.plan = reinterpret_cast<EvictPlan*>(b + w.plan);
  p.mask = reinterpret_cast<uint32_t*>(b + w.mask);
  p.before = reinterpret_cast<int32_t*>(b + w.before);
  p.done = reinterpret_cast<int32_t*>(b + w.done);
  p.status = dev_status;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int vecs = p.kv.row >> 3;
  // 128 bytes where those fill the SMs, else 32: 8 sequences of 520..700 tokens, one layer: 18.7 us with 128 bytes, 16.7 with 32
  const bool narrow = (long long)n * cache->n_layers * ((vecs + 7) / 8) < num_sms();
  const int slices = narrow ? (vecs + 1) / 2 : (vecs + 7) / 8;
  cudaError_t e = launch_k(select_kernel, dim3(n, cache->n_layers), kSelThreads, 0, s, p);
  if (e == cudaSuccess)
    e = launch_k(narrow ? move_kernel<2> : move_kernel<8>, dim3(slices + 1, n, cache->n_layers), kMoveThreads, 0, s, p, slices);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
