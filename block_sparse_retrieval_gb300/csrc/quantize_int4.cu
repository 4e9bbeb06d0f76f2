// quantize_int4.cu -- 4-bit pages: compressing pages, reading them back, appending tokens.
//
// KV-cache survey "大模型推理百倍加速之KV cache篇" lists quantisation of the cache among the
// ways to shrink it; the format and the rounding are in int4_page.cuh (17 408 bytes a
// (page, kv head) slab at d 128, against 65 536 in bf16).
#include "int4_page.cuh"

namespace srkv {
namespace {

constexpr int kInt4Warps = 8;

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t v) {
  return *reinterpret_cast<const __nv_bfloat162*>(&v);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The word (scale, lo) of a row whose values are held 8 per lane by LPR neighbouring lanes.  The
// smallest value and the largest one's negative go round as one pair (NaN wins).
template <int LPR>
__device__ __forceinline__ uint32_t row_word(const int4& w) {
  const uint32_t u[4] = {(uint32_t)w.x, (uint32_t)w.y, (uint32_t)w.z, (uint32_t)w.w};
  __nv_bfloat162 mn = as_bf162(u[0]), mx = mn;
#pragma unroll
  for (int e = 1; e < 4; ++e) {
    mn = __hmin2_nan(mn, as_bf162(u[e]));
    mx = __hmax2_nan(mx, as_bf162(u[e]));
  }
  const uint32_t neg = as_u32(mx) ^ 0x80008000u;
  __nv_bfloat162 both = __hmin2_nan(as_bf162(__byte_perm(as_u32(mn), neg, 0x5410)),
                                    as_bf162(__byte_perm(as_u32(mn), neg, 0x7632)));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1)
    both = __hmin2_nan(both, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(both), o)));
  return int4_row(bf16_lo(as_u32(both)), -bf16_hi(as_u32(both)));
}

// Codes of a lane's 8 values: pair p in the low nibbles of out[p]'s halves.
__device__ __forceinline__ void lane_codes(const int4& w, uint32_t row, uint32_t (&out)[4]) {
  const Int4Coder code(row);
  out[0] = code.pair((uint32_t)w.x);
  out[1] = code.pair((uint32_t)w.y);
  out[2] = code.pair((uint32_t)w.z);
  out[3] = code.pair((uint32_t)w.w);
}

// The key word of a lane's 8 codes.
__device__ __forceinline__ uint32_t key_word(const uint32_t (&c)[4]) {
  return c[0] | (c[1] << 4) | (c[2] << 8) | (c[3] << 12);
}

// Warp = 8 consecutive tokens (an octet) of one listed page and kv head, keys and values: d / 8
// lanes a row with 8 values each (16-byte loads, all issued before the first is used).  A lane's
// 8 key codes are one word.  Value words hold 8 tokens of one element: each lane first joins its
// own tokens' nibbles, pairs of elements in the halves of a register, then the lanes that share
// those elements exchange them, each keeping its share of the words.
// Bytes: 4 d read, d + 8 written a token.  Bound by them at 88 % of the copy peak (4096 pages of 8
// heads, d 128: 459 us); the arithmetic issues on 71 % of the cycles, in pairs of fp32 (one value at
// a time, with rounding and conversion instructions: 930 us).
template <int D>
__global__ void __launch_bounds__(kInt4Warps * 32)
    quantize_int4_kernel(const __nv_bfloat16* __restrict__ k_src,
                         const __nv_bfloat16* __restrict__ v_src, int64_t num_pages,
                         const int32_t* __restrict__ page_ids, int32_t n_pages, int32_t Hkv,
                         unsigned char* __restrict__ kv, int64_t num_slab_pages,
                         const int32_t* __restrict__ slab_ids, int32_t* error_flags) {
  using F = Int4Slab<D>;
  constexpr int LPR = D / 8;      // lanes per row
  constexpr int RPL = 32 / LPR;   // rows per warp-wide load
  constexpr int LOADS = 8 / RPL;
  const int lane = threadIdx.x & 31;
  const int64_t oct = (int64_t)blockIdx.x * kInt4Warps + (threadIdx.x >> 5);
  if (oct >= (int64_t)n_pages * Hkv * (kBlock / 8)) return;
  const int32_t o = (int32_t)(oct % (kBlock / 8));
  const int64_t ih = oct / (kBlock / 8);
  const int32_t i = (int32_t)(ih / Hkv), h = (int32_t)(ih % Hkv);
  const int32_t page = page_ids[i], dst = slab_ids ? slab_ids[i] : page;
  if (page < 0 || (int64_t)page >= num_pages || dst < 0 || (int64_t)dst >= num_slab_pages) {
    if (lane == 0 && o == 0 && h == 0) raise_flags(error_flags, SRKV_EFLAG_PAGE_RANGE);
    return;
  }
  const int sub = lane / LPR, col = (lane % LPR) * 8;  // row within a load, first element
  const int64_t src = (((int64_t)page * Hkv + h) * kBlock + o * 8) * D;
  unsigned char* slab = kv + ((int64_t)dst * Hkv + h) * F::kBytes;
  int4 kw[LOADS], vw[LOADS];
#pragma unroll
  for (int l = 0; l < LOADS; ++l) {
    const int64_t at = src + (int64_t)(l * RPL + sub) * D + col;
    kw[l] = *reinterpret_cast<const int4*>(k_src + at);
    vw[l] = *reinterpret_cast<const int4*>(v_src + at);
  }
  uint32_t* k_words = reinterpret_cast<uint32_t*>(slab);
  uint32_t* v_words = reinterpret_cast<uint32_t*>(slab + F::kVCodes);
  uint32_t* k_rows = reinterpret_cast<uint32_t*>(slab + F::kKRows);
  uint32_t* v_rows = reinterpret_cast<uint32_t*>(slab + F::kVRows);
  // part[p]: elements 2p (low half) and 2p + 1, this lane's tokens j at bit 4 (j / 2)
  uint32_t part[4] = {};
#pragma unroll
  for (int l = 0; l < LOADS; ++l) {
    const int j = l * RPL + sub, tok = o * 8 + j;
    uint32_t c[4];
    uint32_t row = row_word<LPR>(kw[l]);
    lane_codes(kw[l], row, c);
    k_words[tok * F::kWordsPerRow + col / 8] = key_word(c);
    if (col == 0) k_rows[tok] = row;
    row = row_word<LPR>(vw[l]);
    lane_codes(vw[l], row, c);
#pragma unroll
    for (int p = 0; p < 4; ++p) part[p] |= c[p] << (4 * (l * RPL / 2));
    if (col == 0) v_rows[tok] = row;
  }
  int first = 0;  // first of the lane's elements, relative to col
  if constexpr (RPL == 4) {  // tokens 2, 3, 6, 7 sit with the lanes 16 further on
    const bool upper = (lane & 16) != 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) part[p] <<= upper ? 4 : 0;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t send = upper ? part[p] : part[p + 2], keep = upper ? part[p + 2] : part[p];
      part[p] = keep | __shfl_xor_sync(0xffffffffu, send, 16);
    }
    first = upper ? 4 : 0;
  }
  // even tokens (low halves of the words) sit with the lanes of even rows, odd ones LPR further on
  constexpr int kOwn = RPL == 4 ? 1 : 2;  // pairs of elements a lane keeps
  const bool odd = (sub & 1) != 0;
  uint32_t word[2 * kOwn];
#pragma unroll
  for (int p = 0; p < kOwn; ++p) {
    const uint32_t send = odd ? part[p] : part[p + kOwn], keep = odd ? part[p + kOwn] : part[p];
    const uint32_t got = __shfl_xor_sync(0xffffffffu, send, LPR);
    const uint32_t even_tokens = odd ? got : keep, odd_tokens = odd ? keep : got;
    word[2 * p] = __byte_perm(even_tokens, odd_tokens, 0x5410);
    word[2 * p + 1] = __byte_perm(even_tokens, odd_tokens, 0x7632);
  }
  first += odd ? 2 * kOwn : 0;
  uint32_t* vd = v_words + int4_v_word<D>(o * 8, col + first);
  if constexpr (RPL == 2)
    *reinterpret_cast<uint4*>(vd) = make_uint4(word[0], word[1], word[2], word[3]);
  else
    *reinterpret_cast<uint2*>(vd) = make_uint2(word[0], word[1]);
}

// bf16 pair code * scale + lo of the pair of codes in the low nibbles of x's halves: 128 + code is
// a bf16 of its own (0x4300 | code), the subtraction is exact and the multiply-add rounds once.
__device__ __forceinline__ uint32_t pair_values(uint32_t x, __nv_bfloat162 scale,
                                                __nv_bfloat162 lo) {
  const __nv_bfloat162 c = __hsub2(as_bf162((x & 0x000f000fu) | 0x43004300u),
                                   as_bf162(0x43004300u));
  return as_u32(__hfma2(c, scale, lo));
}

// Warp = 16 consecutive tokens of one listed page and kv head.  Keys: d / 8 lanes a row, one word
// in and 16 bytes out a lane.  Values: a lane takes 8 elements of an octet (two 16-byte loads),
// and its 8 words hold 8 tokens of them: 16 bytes out a token.  Every store of a warp covers
// whole rows.  Bytes: d + 8 read, 4 d written a token; bound by them (4096 pages: 404 us, 99 % of
// the copy peak).  Launched so that its set-up overlaps the previous kernel's end: 37 pages of 3
// heads, d 64, 2.91 -> 2.57 us (the quantiser so: 3.00 -> 2.65, but 32 pages of 8 heads 6.06 -> 6.74).
template <int D>
__global__ void __launch_bounds__(kInt4Warps * 32)
    dequantize_int4_kernel(const unsigned char* __restrict__ kv, int64_t num_slab_pages,
                           const int32_t* __restrict__ slab_ids, int32_t n_pages, int32_t Hkv,
                           __nv_bfloat16* __restrict__ k_dst, __nv_bfloat16* __restrict__ v_dst,
                           int64_t num_pages, const int32_t* __restrict__ page_ids,
                           int32_t* error_flags) {
  using F = Int4Slab<D>;
  constexpr int LPR = D / 8;     // lanes per row
  constexpr int RPL = 32 / LPR;  // rows (keys) or octets (values) at once
  constexpr int kToks = 8 * RPL;  // tokens per warp: 16 (d 128) or 32 (d 64)
  const int lane = threadIdx.x & 31;
  const int64_t gw = (int64_t)blockIdx.x * kInt4Warps + (threadIdx.x >> 5);
  griddep_wait();  // programmatic launch: the inputs may be the previous kernel's outputs
  griddep_launch_dependents();
  if (gw >= (int64_t)n_pages * Hkv * (kBlock / kToks)) return;
  const int32_t t0 = (int32_t)(gw % (kBlock / kToks)) * kToks;
  const int64_t ih = gw / (kBlock / kToks);
  const int32_t i = (int32_t)(ih / Hkv), h = (int32_t)(ih % Hkv);
  const int32_t src = slab_ids[i], page = page_ids ? page_ids[i] : src;
  if (src < 0 || (int64_t)src >= num_slab_pages || page < 0 || (int64_t)page >= num_pages) {
    if (lane == 0 && t0 == 0 && h == 0) raise_flags(error_flags, SRKV_EFLAG_PAGE_RANGE);
    return;
  }
  const unsigned char* slab = kv + ((int64_t)src * Hkv + h) * F::kBytes;
  const uint32_t* k_words = reinterpret_cast<const uint32_t*>(slab);
  const uint32_t* v_words = reinterpret_cast<const uint32_t*>(slab + F::kVCodes);
  const uint32_t* k_rows = reinterpret_cast<const uint32_t*>(slab + F::kKRows);
  const uint32_t* v_rows = reinterpret_cast<const uint32_t*>(slab + F::kVRows);
  const int sub = lane / LPR, col = (lane % LPR) * 8;
  const int64_t out = (((int64_t)page * Hkv + h) * kBlock + t0) * D + col;
  const int ot = t0 + 8 * sub;  // the lane's octet of values
  uint32_t kx[8], kr[8], vr[8];
#pragma unroll
  for (int l = 0; l < 8; ++l) {
    const int tok = t0 + l * RPL + sub;
    kx[l] = k_words[tok * F::kWordsPerRow + col / 8];
    kr[l] = k_rows[tok];
    vr[l] = v_rows[ot + l];
  }
  const uint4 va = *reinterpret_cast<const uint4*>(v_words + int4_v_word<D>(ot, col));
  const uint4 vb = *reinterpret_cast<const uint4*>(v_words + int4_v_word<D>(ot, col + 4));
  auto scale2 = [](uint32_t row) { return as_bf162(__byte_perm(row, row, 0x1010)); };
  auto lo2 = [](uint32_t row) { return as_bf162(__byte_perm(row, row, 0x3232)); };
#pragma unroll
  for (int l = 0; l < 8; ++l) {
    const __nv_bfloat162 s = scale2(kr[l]), m = lo2(kr[l]);
    *reinterpret_cast<uint4*>(k_dst + out + (int64_t)(l * RPL + sub) * D) =
        make_uint4(pair_values(kx[l], s, m), pair_values(kx[l] >> 4, s, m),
                   pair_values(kx[l] >> 8, s, m), pair_values(kx[l] >> 12, s, m));
  }
  const uint32_t v[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
#pragma unroll
  for (int j = 0; j < 8; j += 2) {  // tokens j and j + 1: the low and high halves at bit 2 j
    const __nv_bfloat162 s0 = scale2(vr[j]), m0 = lo2(vr[j]);
    const __nv_bfloat162 s1 = scale2(vr[j + 1]), m1 = lo2(vr[j + 1]);
    uint32_t a[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t x = v[2 * e] >> (2 * j), y = v[2 * e + 1] >> (2 * j);
      a[e] = pair_values(__byte_perm(x, y, 0x5410), s0, m0);
      b[e] = pair_values(__byte_perm(x, y, 0x7632), s1, m1);
    }
    __nv_bfloat16* p = v_dst + out + (int64_t)(8 * sub + j) * D;
    *reinterpret_cast<uint4*>(p) = make_uint4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<uint4*>(p + D) = make_uint4(b[0], b[1], b[2], b[3]);
  }
}

// CTA (request r, kv head h): the new token's key and value become row L % 128 of page
// block_table[r][L / 128], and the page's representation vector the fp32 mean of its keys as
// they now stand (lo + code * scale over rows [0, L % 128]): the rows say all there is, so a
// token written again, or after the length was set back, gives the same vector.  Thread =
// (row group, word): fixed order of sums.  Bound by its chain of dependent loads (length, page id,
// page): the new rows are loaded beside the length and the page's earlier rows beside their
// quantisation, so the chain has three links (64 requests x 8 heads 4.5 us, 1 request 2.7 us; one
// more link: 5.4 and 4.3).
constexpr int kAppendThreads = 256;

template <int D>
__global__ void __launch_bounds__(kAppendThreads)
    append_kv_int4_kernel(const __nv_bfloat16* __restrict__ k_new,
                          const __nv_bfloat16* __restrict__ v_new, unsigned char* kv,
                          int64_t num_pages, const int32_t* __restrict__ block_table,
                          int32_t max_blocks, const int32_t* __restrict__ seq_lens, int32_t Hkv,
                          float* __restrict__ reps, int32_t* error_flags) {
  using F = Int4Slab<D>;
  constexpr int LPR = D / 8;                     // words (and lanes) per row
  constexpr int kGroups = kAppendThreads / LPR;  // row groups
  constexpr int kRows = kBlock / kGroups;        // rows per thread at most
  __shared__ float part[kGroups][D];
  __shared__ uint32_t new_k[LPR], new_row;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t r = blockIdx.x / Hkv, h = blockIdx.x % Hkv;
  griddep_wait();  // programmatic launch: the inputs may be the previous kernel's outputs
  griddep_launch_dependents();
  const int32_t L = seq_lens[r];
  int4 x = make_int4(0, 0, 0, 0);
  const int col = (lane % LPR) * 8;
  if (warp < 2)  // warp 0: the key, warp 1: the value; lanes past the row repeat it
    x = *reinterpret_cast<const int4*>((warp ? v_new : k_new) + ((int64_t)r * Hkv + h) * D + col);
  if (L < 0 || (int64_t)L >= (int64_t)max_blocks * kBlock) {
    if (tid == 0 && h == 0) raise_flags(error_flags, SRKV_EFLAG_SEQ_LEN);
    return;
  }
  const int32_t page = block_table[(int64_t)r * max_blocks + L / kBlock];
  if (page < 0 || (int64_t)page >= num_pages) {
    if (tid == 0 && h == 0) raise_flags(error_flags, SRKV_EFLAG_PAGE_RANGE);
    return;
  }
  const int32_t tok = L % kBlock;
  unsigned char* slab = kv + ((int64_t)page * Hkv + h) * F::kBytes;
  uint32_t* k_words = reinterpret_cast<uint32_t*>(slab);
  uint32_t* v_words = reinterpret_cast<uint32_t*>(slab + F::kVCodes);
  uint32_t* k_rows = reinterpret_cast<uint32_t*>(slab + F::kKRows);
  uint32_t* v_rows = reinterpret_cast<uint32_t*>(slab + F::kVRows);
  // the earlier rows of the page (row tok comes from shared memory)
  const int wi = tid % LPR, grp = tid / LPR;
  uint32_t words[kRows], rows[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int t = grp + i * kGroups;
    words[i] = t < tok ? k_words[t * LPR + wi] : 0u;
    rows[i] = t < tok ? k_rows[t] : 0u;
  }
  if (warp < 2) {
    uint32_t* p = v_words + int4_v_word<D>(tok, col);  // elements col .. + 3; the next 4 16 words on
    uint4 va, vb;
    if (warp == 1) {
      va = *reinterpret_cast<const uint4*>(p);
      vb = *reinterpret_cast<const uint4*>(p + 16);
    }
    const uint32_t row = row_word<LPR>(x);
    uint32_t c[4];
    lane_codes(x, row, c);
    if (lane < LPR) {
      if (warp == 0) {
        const uint32_t word = key_word(c);
        k_words[tok * LPR + lane] = word;
        new_k[lane] = word;
        if (lane == 0) {
          k_rows[tok] = row;
          new_row = row;
        }
      } else {
        const int sh = int4_shift(tok & 7);
        auto put = [&](uint32_t w, uint32_t code) { return (w & ~(15u << sh)) | (code << sh); };
        *reinterpret_cast<uint4*>(p) = make_uint4(put(va.x, c[0] & 15u), put(va.y, c[0] >> 16),
                                                  put(va.z, c[1] & 15u), put(va.w, c[1] >> 16));
        *reinterpret_cast<uint4*>(p + 16) = make_uint4(put(vb.x, c[2] & 15u), put(vb.y, c[2] >> 16),
                                                       put(vb.z, c[3] & 15u), put(vb.w, c[3] >> 16));
        if (lane == 0) v_rows[tok] = row;
      }
    }
  }
  __syncthreads();
  float acc[8] = {};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int t = grp + i * kGroups;
    if (t <= tok) {
      const uint32_t w = t == tok ? new_k[wi] : words[i], row = t == tok ? new_row : rows[i];
      const float s = int4_scale(row), lo = int4_lo(row);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += fmaf((float)((w >> int4_shift(e)) & 15u), s, lo);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) part[grp][wi * 8 + e] = acc[e];
  __syncthreads();
  if (tid < D) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) s += part[g][tid];
    reps[((int64_t)page * Hkv + h) * D + tid] = s / (float)(tok + 1);
  }
}

unsigned blocks_of(int64_t warps) { return (unsigned)((warps + kInt4Warps - 1) / kInt4Warps); }

}  // namespace

cudaError_t launch_quantize_int4(const srkv_config& cfg, const void* k_src, const void* v_src,
                                 int64_t num_pages, const int32_t* page_ids, int32_t n_pages,
                                 void* kv, int64_t num_slab_pages, const int32_t* slab_ids,
                                 int32_t* error_flags, cudaStream_t stream) {
  const int32_t Hkv = cfg.num_kv_heads;
  const int64_t warps = (int64_t)n_pages * Hkv * (kBlock / 8);
  if (warps / kInt4Warps >= INT32_MAX) return cudaErrorInvalidValue;
  const auto* k = static_cast<const __nv_bfloat16*>(k_src);
  const auto* v = static_cast<const __nv_bfloat16*>(v_src);
  auto* out = static_cast<unsigned char*>(kv);
  if (cfg.head_dim == 128)
    quantize_int4_kernel<128><<<blocks_of(warps), kInt4Warps * 32, 0, stream>>>(
        k, v, num_pages, page_ids, n_pages, Hkv, out, num_slab_pages, slab_ids, error_flags);
  else
    quantize_int4_kernel<64><<<blocks_of(warps), kInt4Warps * 32, 0, stream>>>(
        k, v, num_pages, page_ids, n_pages, Hkv, out, num_slab_pages, slab_ids, error_flags);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_int4(const srkv_config& cfg, const void* kv, int64_t num_slab_pages,
                                   const int32_t* slab_ids, int32_t n_pages, void* k_dst,
                                   void* v_dst, int64_t num_pages, const int32_t* page_ids,
                                   int32_t* error_flags, cudaStream_t stream) {
  const int32_t Hkv = cfg.num_kv_heads;
  const int64_t warps = (int64_t)n_pages * Hkv * (kBlock / (8 * 256 / cfg.head_dim));
  if (warps / kInt4Warps >= INT32_MAX) return cudaErrorInvalidValue;
  const auto* in = static_cast<const unsigned char*>(kv);
  auto* k = static_cast<__nv_bfloat16*>(k_dst);
  auto* v = static_cast<__nv_bfloat16*>(v_dst);
  const dim3 grid(blocks_of(warps)), block(kInt4Warps * 32);
  return cfg.head_dim == 128
             ? launch_pdl(dequantize_int4_kernel<128>, grid, block, 0, stream, in, num_slab_pages,
                          slab_ids, n_pages, Hkv, k, v, num_pages, page_ids, error_flags)
             : launch_pdl(dequantize_int4_kernel<64>, grid, block, 0, stream, in, num_slab_pages,
                          slab_ids, n_pages, Hkv, k, v, num_pages, page_ids, error_flags);
}

cudaError_t launch_append_kv_int4(const srkv_config& cfg, const void* k_new, const void* v_new,
                                  void* kv, int64_t num_pages, const int32_t* block_table,
                                  int32_t max_blocks, const int32_t* seq_lens, int32_t batch,
                                  float* reps, int32_t* error_flags, cudaStream_t stream) {
  const int32_t Hkv = cfg.num_kv_heads;
  const dim3 grid((unsigned)((int64_t)batch * Hkv)), block(kAppendThreads);
  const auto* k = static_cast<const __nv_bfloat16*>(k_new);
  const auto* v = static_cast<const __nv_bfloat16*>(v_new);
  auto* out = static_cast<unsigned char*>(kv);
  return cfg.head_dim == 128
             ? launch_pdl(append_kv_int4_kernel<128>, grid, block, 0, stream, k, v, out, num_pages,
                          block_table, max_blocks, seq_lens, Hkv, reps, error_flags)
             : launch_pdl(append_kv_int4_kernel<64>, grid, block, 0, stream, k, v, out, num_pages,
                          block_table, max_blocks, seq_lens, Hkv, reps, error_flags);
}

}  // namespace srkv
