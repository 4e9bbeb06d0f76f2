// decode_int4.cuh -- the consumer warps' loop of the decode over 4-bit pages (int4_page.cuh).
//
// softmax(q K^T / sqrt(d)) V with K = klo_t + ks_t ck_td and V = vlo_t + vs_t cv_td (token t, element
// d, codes c in 0..15):
//   logit_t = ks_t (sum_d q_d ck_td) + klo_t (sum_d q_d),
//   out_d   = sum_t (w_t vs_t) cv_td + sum_t w_t vlo_t,     w_t = softmax weight,
// so both products take the bare codes and a row's scale and minimum enter once per (token, head).
// What bounds it: per token and kv head 136 bytes arrive (d 128) and 256 codes have to become
// matrix operands, so a code may cost a few instructions of an SM's 4 a cycle and no more.  A
// code costs 5/8 of one here: a word masked with 0x000f000f or 0x00f000f0 is two fp16 subnormals,
// code * 2^-24 or code * 2^-20, operands of m16n8k16 products as they are (subnormals are
// exact there), and one shift per word reaches the other four.  The powers of two are taken out of
// the query (16 times smaller at the second kind's elements) and of the weights likewise.
//
// A page is 4 groups of 32 tokens, a warp takes kTok of them and a page kGroupWarps warps; the
// CTA's 8 warps work on kGroups consecutive stages at once.  Lane (g, t) of a warp (g = lane / 4):
//   S^T = K . Q^T, two 16-token tiles j per 32 tokens: tile row m holds token 8 (m / 2) + 4 j + (m & 1)
//     for m < 8 and that + 2 for row m + 8, so that rows 2t, 2t + 1, 2t + 8, 2t + 9 are the four
//     tokens whose nibbles sit in bits 8j .. 8j + 7 of both halves of octet t's value words: the
//     weights of S^T feed O^T = V^T . P without moving between lanes but for one movmatrix each;
//   V^T: lane (g, t) reads the words of octet t for elements 4g + 32x .. + 3 (one 16-byte load), two
//     to a 16-row tile.
// Both layouts make every 8-lane phase of the 16-byte shared loads contiguous (128 bytes).
//
// Online softmax with a lazy reference: the weights are 2^(s - m) for a reference m that is raised
// only when some s + log2 vs exceeds it by 2^8, which a vote finds; then the accumulators are
// rescaled.  log2 vs is in it so that the weight times scale that enters the second product as fp16
// stays within its range whatever the values' magnitude (up to 2^8 * 64).
#pragma once

#include "decode_mma.cuh"

namespace srkv {

constexpr float kInt4Headroom = 8.f;       // log2 of the most a weight may exceed its reference
constexpr float kInt4PScale = 64.f;        // on the fp16 weights: 2^(8 + 6) < 65504
constexpr float kInt4VScaleLog2Max = 30.f;  // log2 vs is taken within +-30 in the reference

template <int D, typename WritePartial>
__device__ __forceinline__ void consumer_loop_int4(const DecodeArgs& a, unsigned char* smem,
                                                   int lane, int warp,
                                                   WritePartial&& write_partial) {
  using C = Cfg<D, kInt4Pages>;
  using F = Int4Slab<D>;
  constexpr int kGroupWarps = 2;                       // warps per page
  constexpr int kGroups = kConsumerWarps / kGroupWarps;  // pages at once
  constexpr int kTok = kBlock / kGroupWarps;           // tokens per warp and page
  constexpr int NW = kTok / 32;                        // 32-token groups per warp
  constexpr int KW = D / 32;                           // key words per lane and row
  constexpr int VX = D / 32;                           // 16-byte value loads per lane and octet
  float* sMerge = reinterpret_cast<float*>(smem + C::kOffMerge);
  StageInfo* sInfo = reinterpret_cast<StageInfo*>(smem + C::kOffInfo);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + 2 * C::kStages;
  uint64_t* mb_w1 = empty + C::kStages;
  uint64_t* mb_w2 = mb_w1 + 1;
  uint64_t* mb_r2 = mb_w1 + 2;
  const Lane ln{lane >> 2, lane & 3};
  const int group = warp / kGroupWarps, row0 = (warp % kGroupWarps) * kTok;
  const int tile_row = 8 * (ln.g >> 1) + (ln.g & 1);  // token of tile row g within 32 tokens
  SoftmaxState<D> st;
  st.reset();
  float pm[2] = {0.f, 0.f};  // sum of weight * vlo, heads 2t and 2t + 1 (this lane's tokens)
  uint32_t qb[KW][2][2];     // [word][bits 0..7, 8..15 of its halves][codes * 2^-24, * 2^-20]
#pragma unroll
  for (int i = 0; i < KW; ++i) qb[i][0][0] = qb[i][0][1] = qb[i][1][0] = qb[i][1][1] = 0u;
  float qs = 0.f;            // what the integer-like logits are to be multiplied by (log2 domain)
  float qm0 = 0.f, qm1 = 0.f;  // sum_d q_d of heads 2t, 2t + 1 (log2 domain)
  bool abort = false;
  int32_t merges = 0;

  // End of a segment: reduce the per-lane sums, merge the 8 warps, write the partial.
  auto close_segment = [&](const StageInfo& inf) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], o);
      st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], o);
      pm[0] += __shfl_xor_sync(0xffffffffu, pm[0], o);
      pm[1] += __shfl_xor_sync(0xffffffffu, pm[1], o);
    }
    // only NaN rows seen: a finite reference, so that the merges do not take the part for empty
    if (st.m[0] == -INFINITY && !(st.l[0] == 0.f)) st.m[0] = 0.f;
    if (st.m[1] == -INFINITY && !(st.l[1] == 0.f)) st.m[1] = 0.f;
    constexpr float kUnit = 16777216.f / kInt4PScale;  // 2^24 of the subnormals
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) st.acc[i][c] = fmaf(st.acc[i][c], kUnit, pm[c & 1]);
    const uint32_t ph = (uint32_t)(merges & 1);
    if (warp >= 4) {
      if (merges > 0 && !mbar_wait(mb_r2, ph ^ 1u)) abort = true;
      st.store(sMerge + (warp - 4) * C::kMergeSlot, lane);
      warp_arrive(mb_w1);
    } else {
      if (!mbar_wait(mb_w1, ph)) abort = true;
      st.merge_from(sMerge + warp * C::kMergeSlot, lane);
      if (warp >= 1) {
        st.store(sMerge + warp * C::kMergeSlot, lane);
        warp_arrive(mb_w2);
      } else {
        if (!mbar_wait(mb_w2, ph)) abort = true;
        for (int w = 1; w < 4; ++w) st.merge_from(sMerge + w * C::kMergeSlot, lane);
        warp_arrive(mb_r2);
        write_partial(st, inf, ln);
      }
    }
    ++merges;
  };

  // The unit's query: fp16 with one power of two for all of its heads, the largest magnitude
  // put into [2^14, 2^15), so that bf16's 8 significant bits stay exact down to 2^-25 of it.
  auto load_query = [&](const unsigned char* q) {
    constexpr int QV = D / 32;  // 16-byte loads: elements (D / 4) t .. of head g
    int4 w[QV];
    uint32_t top = 0u;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < QV; ++i) {
      w[i] = ln.g < a.G ? lds128(q + ((size_t)ln.g * D + (D / 4) * ln.t + 8 * i) * 2)
                        : make_int4(0, 0, 0, 0);
      const uint32_t u[4] = {(uint32_t)w[i].x, (uint32_t)w[i].y, (uint32_t)w[i].z,
                             (uint32_t)w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = (u[e] << 16) & 0x7fffffffu, y = u[e] & 0x7fff0000u;
        if (x < 0x7f800000u) top = max(top, x);  // the largest finite magnitude
        if (y < 0x7f800000u) top = max(top, y);
        sum += bf16_lo(u[e]) + bf16_hi(u[e]);
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    qm0 = __shfl_sync(0xffffffffu, sum, 8 * ln.t) * a.scale_log2;      // head 2t
    qm1 = __shfl_sync(0xffffffffu, sum, 8 * ln.t + 4) * a.scale_log2;  // head 2t + 1
    int e = (int)(top >> 23) - 127;        // floor(log2 top), -127 for zeros and subnormals
    e = min(max(e, -112), 100);
    const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    qs = __uint_as_float((uint32_t)(127 + 10 + e) << 23) * a.scale_log2;  // 2^(24 - 14 + e)
#pragma unroll
    for (int i = 0; i < QV; ++i) {
      const uint32_t u[4] = {(uint32_t)w[i].x, (uint32_t)w[i].y, (uint32_t)w[i].z,
                             (uint32_t)w[i].w};
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // the pair in nibble p of both halves
        const float fp = (p & 1) ? f * 0.0625f : f;
        qb[i][p >> 1][p & 1] = pack_f16(bf16_lo(u[p]) * fp, bf16_hi(u[p]) * fp);
      }
    }
  };

  for (int64_t it = 0;; ++it) {
    const int s = (int)(it % C::kStages);
    if (!mbar_wait(&full[s], (uint32_t)((it / C::kStages) & 1))) {
      if (lane == 0) raise_flags(a.error_flags, SRKV_EFLAG_TIMEOUT);
      break;
    }
    const StageInfo inf = sInfo[s];
    if (inf.flags & kLast) {  // the sentinel; it may close the last segment
      if (inf.flags & kSegEnd) {
        close_segment(inf);
        if (abort && lane == 0) raise_flags(a.error_flags, SRKV_EFLAG_TIMEOUT);
      }
      break;
    }
    if (inf.flags & kNewUnit) {
      st.reset();
      pm[0] = pm[1] = 0.f;
      load_query(smem + C::kOffQ + (size_t)s * C::kQBytes);
    }
    if ((int)(it % kGroups) == group && row0 < inf.hi && row0 + kTok > inf.lo) {
      const unsigned char* slab = smem + C::kOffK + (size_t)s * C::kSlab;
      const uint32_t* k_rows = reinterpret_cast<const uint32_t*>(slab + F::kKRows);
      const uint32_t* v_rows = reinterpret_cast<const uint32_t*>(slab + F::kVRows);
      constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
      // ---- logits (log2 domain) of the warp's tokens: [32 tokens][tile][row g: heads 2t, 2t+1,
      //      row g + 8: the same]; vs and vlo of those rows
      float z[NW][2][4], vs[NW][2][2], vl[NW][2][2];
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int ra = row0 + 32 * w + tile_row + 4 * j, rb = ra + 2;
          uint32_t ka[KW], kb[KW];
          if constexpr (KW == 4) {
            const int4 x = lds128(slab + ra * (D / 2) + ln.t * 16);
            const int4 y = lds128(slab + rb * (D / 2) + ln.t * 16);
            ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
            kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
          } else {
            const int2 x = *reinterpret_cast<const int2*>(slab + ra * (D / 2) + ln.t * 8);
            const int2 y = *reinterpret_cast<const int2*>(slab + rb * (D / 2) + ln.t * 8);
            ka[0] = x.x, ka[1] = x.y;
            kb[0] = y.x, kb[1] = y.y;
          }
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < KW; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint32_t x = ka[i] >> (8 * p), y = kb[i] >> (8 * p);
              mma_16816_f16(acc, x & kLow, y & kLow, x & kHigh, y & kHigh, qb[i][p][0],
                            qb[i][p][1]);
            }
          const uint32_t pa = k_rows[ra], pb = k_rows[rb], va = v_rows[ra], vb = v_rows[rb];
          const float fa = int4_scale(pa) * qs, fb = int4_scale(pb) * qs;
          z[w][j][0] = fmaf(acc[0], fa, int4_lo(pa) * qm0);
          z[w][j][1] = fmaf(acc[1], fa, int4_lo(pa) * qm1);
          z[w][j][2] = fmaf(acc[2], fb, int4_lo(pb) * qm0);
          z[w][j][3] = fmaf(acc[3], fb, int4_lo(pb) * qm1);
          vs[w][j][0] = int4_scale(va);
          vs[w][j][1] = int4_scale(vb);
          vl[w][j][0] = int4_lo(va);
          vl[w][j][1] = int4_lo(vb);
        }
      // ---- rows that are not attended: weight 0, and their parameters are not data
      const bool whole = inf.lo <= row0 && inf.hi >= row0 + kTok &&
                         (inf.ie >= row0 + kTok || inf.ws <= row0 || inf.ws <= inf.ie);
      if (!whole) {
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int r = row0 + 32 * w + tile_row + 4 * j + 2 * x;
              if (!(r >= inf.lo && r < inf.hi && (r < inf.ie || r >= inf.ws))) {
                z[w][j][2 * x] = z[w][j][2 * x + 1] = -INFINITY;
                vs[w][j][x] = vl[w][j][x] = 0.f;
              }
            }
      }
      // ---- raise the reference if some weight would pass its headroom
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float lv = fminf(fmaxf(__log2f(vs[w][j][x]), -kInt4VScaleLog2Max),
                                   kInt4VScaleLog2Max);
            mx0 = fmaxf(mx0, z[w][j][2 * x] + lv);
            mx1 = fmaxf(mx1, z[w][j][2 * x + 1] + lv);
          }
      if (__any_sync(0xffffffffu,
                     mx0 > st.m[0] + kInt4Headroom || mx1 > st.m[1] + kInt4Headroom)) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        const float n0 = fmaxf(st.m[0], mx0), n1 = fmaxf(st.m[1], mx1);
        const float a0 = n0 == -INFINITY ? 1.f : fast_exp2(st.m[0] - n0);
        const float a1 = n1 == -INFINITY ? 1.f : fast_exp2(st.m[1] - n1);
        st.m[0] = n0;
        st.m[1] = n1;
        st.l[0] *= a0;
        st.l[1] *= a1;
        pm[0] *= a0;
        pm[1] *= a1;
#pragma unroll
        for (int i = 0; i < C::MT; ++i) {
          st.acc[i][0] *= a0;
          st.acc[i][1] *= a1;
          st.acc[i][2] *= a0;
          st.acc[i][3] *= a1;
        }
      }
      const float base0 = st.m[0] == -INFINITY ? 0.f : st.m[0];
      const float base1 = st.m[1] == -INFINITY ? 0.f : st.m[1];
      // ---- weights and O^T += V^T . P
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        uint32_t b[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float e0 = fast_exp2(z[w][j][0] - base0), e1 = fast_exp2(z[w][j][1] - base1);
          const float e2 = fast_exp2(z[w][j][2] - base0), e3 = fast_exp2(z[w][j][3] - base1);
          st.l[0] += e0 + e2;
          st.l[1] += e1 + e3;
          pm[0] = fmaf(e0, vl[w][j][0], fmaf(e2, vl[w][j][1], pm[0]));
          pm[1] = fmaf(e1, vl[w][j][0], fmaf(e3, vl[w][j][1], pm[1]));
          // fp16 weights (half a step is 2^-12 of each, independent over the tokens); the rows
          // g + 8 meet the codes * 2^-20
          const float fa = vs[w][j][0] * kInt4PScale, fb = vs[w][j][1] * (kInt4PScale / 16.f);
          b[j][0] = movmatrix_trans(pack_f16(e0 * fa, e1 * fa));
          b[j][1] = movmatrix_trans(pack_f16(e2 * fb, e3 * fb));
        }
        const unsigned char* v = slab + F::kVCodes + (row0 / 32 + w) * (D / 4) * 64 + ln.t * 16;
#pragma unroll
        for (int x = 0; x < VX; ++x) {
          const int4 q4 = lds128(v + (ln.g + 8 * x) * 64);
          const uint32_t u[4] = {(uint32_t)q4.x, (uint32_t)q4.y, (uint32_t)q4.z, (uint32_t)q4.w};
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t p = u[2 * h] >> (8 * j), q = u[2 * h + 1] >> (8 * j);
              mma_16816_f16(st.acc[2 * x + h], p & kLow, q & kLow, p & kHigh, q & kHigh, b[j][0],
                            b[j][1]);
            }
        }
      }
    }
    // release the stage
    warp_arrive(&empty[s]);

    if (inf.flags & kSegEnd) {
      close_segment(inf);
      if (abort) {
        if (lane == 0) raise_flags(a.error_flags, SRKV_EFLAG_TIMEOUT);
        break;
      }
    }
  }
}

}  // namespace srkv
