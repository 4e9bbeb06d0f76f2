// int4_page.cuh -- the 4-bit page format: what a slab holds, and how one row becomes codes.
//
// A slab is one (page, kv head): 128 tokens of keys and values.  A row x of d values (one
// token's key or value) is held as 4-bit codes with its own scale and minimum,
//   lo = min x (bf16, exact),  scale = (max x - lo) / 15 rounded up to bf16,
//   code = the integer nearest to (x - lo) / scale (the difference in fp32, ties to even),
// and stands for lo + code * scale.  Rounding the scale up keeps 15 * scale >= max x - lo, so no
// code is clipped; it costs at most 2^-7 of the step.  One scale per row (as the E4M3 pages have)
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

// The row's word from its smallest and largest value (exact bf16 values; NaN or an infinity
// among the row's values shows in one of them).
__device__ __forceinline__ uint32_t int4_row(float lo, float hi) {
  const float s = __fdiv_rn(hi - lo, 15.f);
  const uint32_t up = (__float_as_uint(s) + 0xffffu) & 0xffff0000u;  // s >= 0: towards +inf
  const bool ok = fmaf(15.f, __uint_as_float(up), fabsf(lo)) < INFINITY;  // false for NaN too
  return ok ? (up >> 16) | (__float_as_uint(lo) & 0xffff0000u) : kInt4BadRow;
}

// Code of x in a row of that scale and minimum.  t = (x - lo) * inv (inv = 1 / scale in fp32) is
// within 15 * 2^-22 of the quotient, so its nearest integer c is the quotient's unless the
// quotient lies about half-way between two: then the remainder x - lo - c * scale decides.  It is
// exact in fp32 (a multiple of the difference's last place, no larger than the scale).
__device__ __forceinline__ uint32_t int4_code(float x, float lo, float scale, float inv) {
  const float diff = __fsub_rn(x, lo);
  const float t = __fmul_rn(diff, inv);
  float c = rintf(t);
  if (fabsf(t - c) > 0.4999f) {
    const float r = fmaf(-c, scale, diff), half = 0.5f * scale;
    const bool odd = (int)c & 1;
    if (r > half || (r == half && odd)) c += 1.f;
    if (r < -half || (r == -half && odd)) c -= 1.f;
  }
  c = fminf(fmaxf(c, 0.f), 15.f);  // NaN (a bad row) becomes 0
  return (uint32_t)c;
}

// 1 / scale for int4_code; 0 for a constant or a bad row (every code is then 0).  A scale
// below 2^-126 (only where a row's whole range is below 2^-122) has no finite reciprocal
// of full precision: such a row is taken as constant, off by less than 2^-122.
__device__ __forceinline__ float int4_inv(float scale) {
  return scale >= 1.17549435e-38f ? __fdiv_rn(1.f, scale) : 0.f;
}

}  // namespace srkv
