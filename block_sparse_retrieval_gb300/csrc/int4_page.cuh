// int4_page.cuh -- the 4-bit page format: what a slab holds, and how one row becomes codes.
//
// A slab is one (page, kv head): 128 tokens of keys and values.  A row x of d values (one
// token's key or value) is held as 4-bit codes with its own scale and minimum,
//   lo = min x (bf16, exact),  scale = (max x - lo) / 15 rounded up to bf16,
//   code = the integer nearest to (x - lo) / scale (difference and quotient in fp32, ties to even),
// and stands for lo + code * scale.  Rounding the scale up keeps 15 * scale >= max x - lo, so no
// code is clipped; it costs at most 2^-7 of the step.  (Down where lo + 15 * scale would round past
// bf16's largest value, so that every finite row reads back finite.)  One scale per row (as the E4M3 pages have)
// because a row is what a decode step appends.  A constant row has scale 0.  A row that holds
// an infinity or a NaN, or whose range passes fp32, has scale = lo = NaN: it reads back as
// NaN and is not hidden behind finite codes.
//
// Bytes of a slab, in order (128 d + 1024 in all, so that one bulk copy moves it):
//   keys' codes    [128][d / 8] words: elements 8i .. 8i+7 of a token in word i
//   values' codes  [4][d / 4][4][4] words: word (w, c, t, e) has element 4c + e of tokens
//                  32w + 8t .. 32w + 8t + 7
//   keys' rows     [128] words: scale (low half) and lo (high half), both bf16
//   values' rows   [128] words, the same
// The eight codes of a word run along the axis its matrix product contracts (d for keys, tokens
// for values); code j sits at bit 4 (j / 2) + 16 (j mod 2), so that masking a word with
// 0x000f000f (or 0x00f000f0) leaves a pair of neighbours in its two halves: two fp16 subnormals
// of value code * 2^-24 (code * 2^-20), which the tensor cores take as they are.
#pragma once

#include "srkv_internal.cuh"

namespace srkv {

template <int D>
struct Int4Slab {
  static constexpr int kWordsPerRow = D / 8;
  static constexpr int kVCodes = kBlock * D / 2;        // byte offset of the values' codes
  static constexpr int kKRows = kBlock * D;             // ... of the keys' rows
  static constexpr int kVRows = kKRows + kBlock * 4;    // ... of the values' rows
  static constexpr int kBytes = kVRows + kBlock * 4;
  static_assert(kBytes % 128 == 0, "slabs stay aligned");
};

__host__ __device__ constexpr int64_t int4_slab_bytes(int32_t d) {
  return (int64_t)kBlock * d + 2 * kBlock * 4;
}

// Bit of code j in its word.
__host__ __device__ constexpr int int4_shift(int j) { return 4 * (j >> 1) + 16 * (j & 1); }

// Word index of element e of token `tok` among the values' codes.
template <int D>
__host__ __device__ constexpr int int4_v_word(int tok, int e) {
  return (((tok >> 5) * (D / 4) + (e >> 2)) * 4 + ((tok >> 3) & 3)) * 4 + (e & 3);
}

__device__ __forceinline__ float int4_scale(uint32_t row) { return bf16_lo(row); }
__device__ __forceinline__ float int4_lo(uint32_t row) { return bf16_hi(row); }

constexpr uint32_t kInt4BadRow = 0x7fc07fc0u;  // scale = lo = NaN
constexpr float kPastBf16 = 3.39617752923046e38f;  // 2^128 - 2^119: rounds past bf16's last value

// The row's word from its smallest and largest value (exact bf16 values; NaN or an infinity
// among the row's values shows in one of them).  The scale is the smallest bf16 whose 15-fold (exact
// in fp32) reaches the range: range / 15 cut to bf16, or the next one.  Where that would make the
// row's top read back as infinity, the one below it: the top then lies 15 (1 + 2^-7) < 15.5 steps
// up at most, so that no code passes 15 either.
__device__ __forceinline__ uint32_t int4_row(float lo, float hi) {
  const float range = hi - lo;
  uint32_t s = __float_as_uint(range * (1.f / 15.f)) & 0xffff0000u;
  if (15.f * __uint_as_float(s) < range) s += 0x10000u;
  if (fmaf(15.f, __uint_as_float(s), lo) >= kPastBf16) s -= 0x10000u;
  return range < INFINITY ? (s >> 16) | (__float_as_uint(lo) & 0xffff0000u)  // (NaN: false)
                          : kInt4BadRow;
}

// About 1 / scale (2^-22 off at most); 0 for a constant or a bad row, and for a scale below 2^-126
// (a row whose whole range is below 2^-122: taken as constant).
__device__ __forceinline__ float int4_inv(float scale) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
  return scale >= 1.17549435e-38f ? r : 0.f;
}

// Pairs of fp32 in one 64-bit register: one instruction for both.
struct F32x2 {
  uint64_t v;
  __device__ __forceinline__ F32x2() {}
  __device__ __forceinline__ F32x2(float x, float y) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  }
  __device__ __forceinline__ void get(uint32_t& x, uint32_t& y) const {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(v));
  }
};
__device__ __forceinline__ F32x2 add2(F32x2 a, F32x2 b) {
  F32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F32x2 mul2(F32x2 a, F32x2 b) {
  F32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F32x2 fma2(F32x2 a, F32x2 b, F32x2 c) {
  F32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Codes of rows' values, a pair of bf16 at a time.
struct Int4Coder {
  F32x2 neg_lo, inv, neg_scale;
  uint32_t keep;  // 0 for a bad row
  __device__ __forceinline__ explicit Int4Coder(uint32_t row) {
    const float s = int4_scale(row), lo = int4_lo(row), r = int4_inv(s);
    neg_lo = F32x2(-lo, -lo);
    inv = F32x2(r, r);
    neg_scale = F32x2(-s, -s);
    keep = row == kInt4BadRow ? 0u : 0x000f000fu;
  }
  // The pair's codes in the low nibbles of the result's halves.  t = (x - lo) * inv is a few ulps
  // off the quotient; its remainder (exact) times inv corrects it to the nearest fp32 (Markstein's step,
  // "Computation of elementary functions on the IBM RISC System/6000 processor", 1990), which is the
  // quotient itself where fp32 holds it, a half-way case among them.  Adding 1.5 * 2^23 rounds to an
  // integer, ties to even, and leaves it in the low bits.
  __device__ __forceinline__ uint32_t pair(uint32_t bf16x2) const {
    const F32x2 x(bf16_lo(bf16x2), bf16_hi(bf16x2));
    const F32x2 diff = add2(x, neg_lo);
    F32x2 t = mul2(diff, inv);
    t = fma2(fma2(t, neg_scale, diff), inv, t);
    t = add2(t, F32x2(12582912.f, 12582912.f));
    uint32_t a, b;
    t.get(a, b);
    return __byte_perm(a, b, 0x5410) & keep;
  }
};

}  // namespace srkv
