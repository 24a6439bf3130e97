// Rows of the latent cache in 4 bits: how a row lies in memory, and the way
// between bf16 latents and their codes.
//
//   rank / 2 bytes    codes, E2M1, entry 2c in the low nibble of byte c
//   2 rope bytes      the rotary key, bf16
//   rank / 16 bytes   scales, one per 16 entries: 5 exponent bits (bias 15) and 3
//                     significand bits, no sign; an exponent of 31 is NaN
//   zeros up to a multiple of 16 bytes
//
// A code has 2 significant bits and a scale 4, so every product is a bf16 exactly:
// a row in 4 bits is a bf16 row with other bits, and what reads one expands it
// without a rounding.  Scales of E4M3 (448 down to 2^-9) would want one more
// factor per row or tensor for rows far from 1 in size; with the sign's bit as a
// fifth exponent bit they reach from 2^-17 to 61440 by themselves.
#pragma once

#include "kv_common.cuh"

namespace moe {

constexpr int kFpBlock = 16;             // entries of a scale

// ---------------------------------------------------------------- codes to bf16
// The factor of one block in both halves of a word: 2^6 times the scale.  The byte shifted by 4 is a bf16 of 2^-112 times
// the scale's value (exponent 0 included: both formats' subnormals), so one exact product moves it into place.
__device__ inline uint32_t fp4_factor(uint32_t byte) {
  const uint32_t b = byte << 4;
  uint32_t f;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(f) : "r"(b | b << 16), "r"(0x7A807A80u));   // 2^118
  return byte >= 0xF8u ? 0x7FC07FC0u : f;
}

// Eight codes of a word times their scale, as eight bf16, exactly.  A code's exponent bits and significand bit at bits
// 8..6 of a bf16 are its value times 2^-126; 2^120 and then the factor bring it up without a rounding on the way.
__device__ inline uint4 fp4_expand8(uint32_t w, uint32_t factor) {
  const uint32_t a = w & 0x0F0F0F0Fu, b = (w >> 4) & 0x0F0F0F0Fu;   // entries 2 j, and 2 j + 1, in byte j
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t t;     // bytes: a's, 0, b's, 0 (a selector with bit 3 repeats a sign, here that of a byte below 16)
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(t) : "r"(a), "r"(b), "r"(0x8080u | (uint32_t)j | (4u + j) << 8));
    const uint32_t raw = (t * 0x1040u) & 0x81C081C0u;   // magnitude to bits 6..8, sign to bit 15
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[j]) : "r"(raw), "r"(0x7B807B80u));        // 2^120
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(o[j]) : "r"(factor));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The same with one product a pair, for scales below 4: factor = 2^126 times the scale.
__device__ inline uint4 fp4_expand8_small(uint32_t w, uint32_t factor) {
  const uint32_t a = w & 0x0F0F0F0Fu, b = (w >> 4) & 0x0F0F0F0Fu;
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t t;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(t) : "r"(a), "r"(b), "r"(0x8080u | (uint32_t)j | (4u + j) << 8));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[j]) : "r"((t * 0x1040u) & 0x81C081C0u), "r"(factor));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ inline uint32_t fp4_factor_small(uint32_t scales) {      // of the low byte
  uint32_t b, f;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(b) : "r"(scales), "r"(0x4040u));                      // the byte in both halves
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(f) : "r"(b << 4), "r"(0x7B007B00u));                // 2^119, twice: from 2^-112
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(f) : "r"(0x7B007B00u));
  return f;
}

// Where a thread's quarter of 128 entries of a tile's row lies (16 bytes of codes, 32 entries): four 16-byte columns of a
// K-major tile with the 128-byte swizzle that TMA writes.  Quarter v is half of 64-entry chunk v / 2.  Lanes l, l + 8,
// l + 16, l + 24 have one row, so that the eight lanes of a store phase meet eight rows, whose columns all differ.
struct Fp4Place {
  uint32_t at;       // column 0's address; column i's has bits 4 and 5 flipped by i
  __device__ Fp4Place(uint32_t tile, int chunk_bytes, int row, int v)
      : at(tile + (v >> 1) * chunk_bytes + row * 128 + ((((v & 1) * 4) ^ (row & 7)) << 4)) {}
};

__device__ inline void st_shared_v4(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// The quarter's entries to `to`, `offset` bytes on (a whole warp at once): with one product where all of the warp's scales
// are below 4 (a block whose largest entry is 24, far above a normalised latent), else with two, which also know a scale
// that is NaN.  HALVES: how many halves of the quarter are written out.  The warps that expand share their instruction
// caches with the kernel's other roles: beside the decode kernel's softmax one half in a loop is best (832,000 tokens of 16
// heads 223 us, with both written out 244, with all four quarters of a row 307), in the smaller weights kernel both are (168
// us, one in a loop 177).
template <int HALVES>
__device__ inline void fp4_store32(const Fp4Place& to, uint32_t offset, uint4 c, uint32_t scales) {
  const bool large = (scales & 0xFFu) >= 0x88u || scales >= 0x8800u;
  uint32_t at = to.at + offset;
  if (!__any_sync(0xffffffffu, large)) {
#pragma unroll HALVES
    for (int i = 0; i < 2; ++i) {
      const uint32_t f = fp4_factor_small(scales);
      st_shared_v4(at, fp4_expand8_small(c.x, f));
      st_shared_v4(at ^ 16, fp4_expand8_small(c.y, f));
      c.x = c.z;
      c.y = c.w;
      scales >>= 8;
      at ^= 32;
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      st_shared_v4(at ^ (i << 4), fp4_expand8(c.x, fp4_factor(i < 2 ? scales & 0xFFu : scales >> 8)));
      c.x = c.y;
      c.y = c.z;
      c.z = c.w;
    }
  }
}

// A tile's codes and scales as they come from the pages, `rows` rows: 128-byte pieces of the codes, one region behind the
// other, each with the 128-byte swizzle (eight rows' quarters then lie in different banks), and 32 bytes of scales a row.
__host__ __device__ inline int fp4_regions(int rank) { return (rank / 2 + 127) / 128; }
__host__ __device__ inline int fp4_stage_bytes(int rank, int rows) { return rows * (128 * fp4_regions(rank) + 32); }

// Quarter v of pair j of row r of a stage that begins at `stage`.
__device__ inline void fp4_fetch(uint32_t stage, int rows, int regions, int r, int v, int j, uint4& c, uint32_t& scales) {
  const uint32_t at = stage + (uint32_t)((j >> 1) * rows * 128 + r * 128 + ((((j & 1) * 4 + v) ^ (r & 7)) << 4));
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(c.x), "=r"(c.y), "=r"(c.z), "=r"(c.w) : "r"(at) : "memory");
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(stage + (uint32_t)(regions * rows * 128 + r * 32 + 8 * j + 2 * v)) : "memory");
  scales = x;
}

__device__ inline uint32_t ldg_stream_u16(const void* p) {
  uint16_t v;
  asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

// Between a thread's ordinary writes to shared memory and the tensor cores' reads of them: by the thread that wrote, before
// it signals.
__device__ inline void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------- bf16 to codes
struct Fp4Block {
  uint2 codes;
  uint32_t scale;
  bool clamped;      // the largest scale was too small
};

__device__ inline uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// 16 bf16 values to codes: scale = largest magnitude / 6, rounded to nearest (ties to even); code = value / scale,
// rounded likewise.  A block with a NaN or an infinity becomes NaN.
__device__ inline Fp4Block fp4_quantise(const uint4& lo, const uint4& hi) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_u16x2(top, w[i] & 0x7FFF7FFFu);      // magnitudes order like their bits
  top = max(top & 0xFFFFu, top >> 16);
  Fp4Block q;
  q.codes = make_uint2(0, 0);
  q.clamped = false;
  if (top >= 0x7F80u) {
    q.scale = 0xFFu;
    return q;
  }
  // the quotient's own rounding moves no tie: 5 significant bits times 6 are exact
  const float want = __fdiv_rn(__uint_as_float(top << 16), 6.0f);
  uint32_t s;
  if (want >= 0x1p-14f) {
    const uint32_t b = __float_as_uint(want);
    s = ((b + 0x7FFFFu + (b >> 20 & 1u)) >> 20) - (112u << 3);
    q.clamped = s > 0xF7u;
    s = min(s, 0xF7u);
  } else {
    s = (uint32_t)__float2int_rn(want * 0x1p17f);
  }
  q.scale = s;
  if (s == 0) return q;
  const float scale = s < 8u ? (float)s * 0x1p-17f : __uint_as_float((s + (112u << 3)) << 20);
  const float inv = __frcp_rn(scale);
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x = e ? bf16_hi(w[i]) : bf16_lo(w[i]);
      // x / scale: the remainder's correction makes the quotient exact where it has few bits, so ties stay ties
      const float y = x * inv;
      v[e] = fmaf(fmaf(-y, scale, x), inv, y);
    }
    uint32_t byte;
    asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n cvt.u32.u8 %0, b;\n}\n" : "=r"(byte) : "f"(v[1]), "f"(v[0]));
    c[i >> 2] |= byte << (8 * (i & 3));
  }
  q.codes = make_uint2(c[0], c[1]);
  return q;
}

}  // namespace moe
