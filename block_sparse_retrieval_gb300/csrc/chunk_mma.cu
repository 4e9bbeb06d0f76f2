// chunk_mma.cu -- attention of a chunk over the paged cache on the tensor cores (bf16).
//
// A CTA takes an item: up to 256 rows (two tiles of 128) of one (request, kv head) over a list of pages.  Per
// page and tile:  S = Q K^T (128 x 128, fp32, in tensor memory);  the tile's two warpgroups, two threads a row, read it,
// update the row's maximum and sum, and write P = 2^(c S - R) as bf16 over S;  O += P V (O in tensor memory).
//
//   warps 0-7, 8-15  softmax and output of tile 0, 1: two threads a row, 64 of a page's tokens each
//   warps 16, 17     issue the products of tile 0, 1
//   warp 18          takes items and copies pages (TMA) into a ring of stages: K, V, K, V ...
//   warp 19          copies the queries of the next item once the last product with the present ones is done, and
//                    cleans values (below)
//
// Why so.  256 rows share a page because the copy of a page (64 KB) then takes half the time of its products
// (2048 cycles).  S and O of two tiles fill the 512 columns of tensor memory, so P lies on S and the next S waits for O's
// product: the tiles have to alternate, one's products running while the other is at its exponentials.  Two warps issue
// them, taking turns (in step, 13.5 ms for 8192 of 131072 tokens): waits and releases of one fall into the other's
// block (one warp for both: 11.3 ms; two, in turns: 10.7; told two products ahead: 10.3 to 10.5).  P is handed over in
// two parts, so that its product begins before the last exponential.  One thread a row (128 logits, 208 registers) took
// 12.4 ms, with 168 registers and spills 19.6.
//
// What bounds it.  Long lists at d 128: the tensor cores; 2740 to 2850 cycles a page pair, of which 2048 are products
// (77 % of the cycles by the counters), 1510 to 1657 TFLOP/s (by the GPU's power) = 0.78 to 0.86 of the measured burst
// rate of a library product and 0.88 to 0.96 of the sustained one; what is left is the chain from a product's end
// over the exponentials to the next turn.  At d 64 the softmax warps: 2510 cycles for 1024 of products.  (There S and P
// could lie apart and products run ahead; that put both tiles' exponentials in step: 2685.)  Single tokens: bytes; 64
// of them over windows of 8216 take 304 us, the measured copy rate.  Short lists: an item's start and end
// (queries, first page, output), some 2 us that the next item does not hide.
//
// Rounding.  P is rounded to bf16 (by up to 2^-8 of each weight: the product's operands share a type with V),
// its sum taken before that; S, R, sums and O are fp32.  The reference R that the exponentials subtract follows
// the maximum; in items of two tiles only when that has grown by more than 2^8, as scaling O takes time there that the
// products wait for (prompt of 4096 102 us; at any growth 111, at 2^4 107): sums and outputs are the same for any
// reference, as long as 2^8 times a sum of values stays in fp32.  A weight of exactly 1 is not rounded, so the error
// of outputs against 64 bits (relative, root mean square; the rounding of the output itself 0.0016 to 0.0017)
// is 0.0022 in two tiles, and 0.0018 to 0.0019 in one (0.0020 to 0.0026 with a reference left behind: with few rows it
// hangs on a few large weights).
//
// Hidden tokens.  A weight of zero does not hide a value that is not finite, so the pages of an item that some
// row sees in part are looked through before their product: rows behind the sequence are cleared, and elements of
// tokens hidden from some row that are not finite are replaced by zero and their token noted; the rows that do attend
// such a token get the element back at the end.
#include "chunk_plan.cuh"
#include "tcgen05.cuh"

namespace srkv {

bool encode_cache_map(CUtensorMap* map, const void* base, int64_t num_pages, int32_t Hkv, int32_t d,
                      bool e4m3);
bool encode_rows_map(CUtensorMap* map, const void* q, int64_t tokens, int64_t stride, int32_t heads, int32_t d,
                     int32_t box_heads, int32_t box_tokens);

namespace {

constexpr int kThreads = 640;
constexpr int kMmaWarp = 16, kPageWarp = 18;  // and the helper, the last one
constexpr int kSlots = 3;      // items known at a time
constexpr int kPageInfo = 8;   // pages between their copy and their softmax, at most
constexpr int kParts = 4;      // pages seen in part and not yet multiplied, at most: their stages are not refilled
constexpr int kOdd = 7;        // pages that an item's rows see in part, at most: 3 at each end of a window of 256 rows, 1 at
                               // the first tokens
// Registers: 512 x 104 + 128 x 64 = 640 x 96, what the block is launched with.
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;
constexpr int kTellAhead = 2;  // products of 16 columns before the end of a block at which the other tile's warp is told:
                               // 1, 2, 3, 4 of them 10.5, 10.3, 10.5, 10.9 ms for 8192 of 131072 tokens
constexpr int kPrefetch = 3;   // pages that a CTA asks for while the plan is made
constexpr float kGrow = 8.f;   // log2 of the growth of a maximum that the reference of an item of two tiles lets pass

template <int D>
struct Geo {
  static constexpr int kTileBytes = 128 * D * 2;       // a tile of Q, a page of K or V
  static constexpr int kBlockBytes = 128 * 128;        // its blocks of 64 columns
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kS = 0, kO = 256;          // columns of tensor memory: S0 S1 O0 O1
  static constexpr size_t kOffQ = 0, kOffStage = 2 * kTileBytes,
                          kOffBar = kOffStage + (size_t)kStages * kTileBytes;
};

struct OddPage {
  uint32_t tokens[4];  // those with an element that is not finite
  int32_t block;
};

template <int kStages>
struct Shared {
  uint64_t full[kStages], empty[kStages];
  uint64_t item_full[kSlots], item_empty[kSlots];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2][2], o_full[2];  // P in two parts: the first 32 tokens of each half, the others
  uint64_t pair[2][4];  // the two warps of a tile's 32 rows
  uint64_t v_part[kParts], v_clean[kParts];
  int2 part[kParts];  // stage of a page seen in part, and the parity of its copy
  uint64_t turn[2];  // whose block of products comes next
  uint64_t drain[2];
  ChunkItem item[kSlots];
  int32_t page[kPageInfo];  // 4 block + how it is seen
  float note[2][2][128];  // [tile][half][row]: a maximum, or a sum
  OddPage odd[kSlots][kOdd];
  int32_t n_odd[kSlots];
  uint32_t tmem;
};

enum { kPart = 1, kAbsent = 2 };  // how an item's rows see a page: 0 whole

struct Maps {
  CUtensorMap k, v;
  CUtensorMap q;       // valid where q_box > 0
  int32_t q_box;       // tokens of a tile of 128 rows, where the group divides 128; else 0
};

__device__ __forceinline__ void tma_page(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Counts uses of a ring of N barriers: index, and the parity to wait for (the consumer's; the producer
// waits for the other one, which a fresh barrier passes).
template <int N>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ Ring plus(int n) const {  // n < N
    Ring r = {at + n, phase};
    if (r.at >= N) {
      r.at -= N;
      r.phase ^= 1;
    }
    return r;
  }
  __device__ __forceinline__ void skip(int32_t n) {
    const int32_t to = at + n;
    phase ^= (uint32_t)(to / N) & 1;
    at = to % N;
  }
};

__device__ __forceinline__ int32_t page_of(const ChunkItem& it, int32_t j) {
  return j < it.na ? j : j + it.shift;
}

__device__ __forceinline__ void item_span(const ChunkItem& it, const DivideBy& by_group, int32_t& p_lo,
                                          int32_t& p_hi) {
  p_lo = it.p0 + (int32_t)by_group.div(it.row0);
  p_hi = it.p0 + (int32_t)by_group.div(it.row0 + it.rows - 1);
}

// 32 rows of V in shared memory, of a page that some row sees in part; `behind`: the lane's row is behind the
// sequence and is cleared; `scan`: it is hidden from some row and not from all, and its elements that are not finite
// are replaced by zero.  Returns (in every lane) the rows that had one.
template <int D>
__device__ __forceinline__ uint32_t clean_values(unsigned char* rows, bool behind, bool scan, int lane) {
  // a lane's row is 128 bytes of each block of 64 columns; the lanes start at different 16-byte chunks
  const uint32_t row = smem_u32(rows) + lane * 128 + (lane & 7) * 16;
  if (behind) {
#pragma unroll 1
    for (int b = 0; b < D / 64; ++b)
#pragma unroll
      for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"((row ^ (c * 16)) + b * (128 * 128)), "r"(0)
                     : "memory");
  }
  if (!__any_sync(0xffffffffu, scan)) return 0;
  // zero times an element added up: NaN if one is not finite
  uint32_t odd[4] = {0, 0, 0, 0};
#pragma unroll 1
  for (int b = 0; b < D / 64; ++b) {
    uint32_t w[8][4];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[c][0]), "=r"(w[c][1]), "=r"(w[c][2]), "=r"(w[c][3])
                   : "r"((row ^ (c * 16)) + b * (128 * 128)));
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(odd[i]) : "r"(w[c][i]), "r"(0));
  }
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= (((odd[i] & 0x7fff7fffu) + 0x007f007fu) & 0x80008000u) != 0;
  any = any && scan;
  if (any) {
    uint4* at = reinterpret_cast<uint4*>(rows + lane * 128);
#pragma unroll 1
    for (int c = 0; c < D / 8; ++c) {
      uint4& x = at[(c / 8) * (128 * 128 / 16) + c % 8];
      uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((v[i] & 0x7f80u) == 0x7f80u) v[i] &= 0xffff0000u;
        if ((v[i] & 0x7f800000u) == 0x7f800000u) v[i] &= 0xffffu;
      }
      x = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  return __ballot_sync(0xffffffffu, any);
}

// What clean_values took out of element `col` of the values that a row at `pos` attends.
__device__ __forceinline__ float odd_value(const ChunkArgs& a, int32_t request, int32_t head, const OddPage* odd,
                                           int n, int32_t pos, int col) {
  float x = 0.f;
  for (int i = 0; i < n; ++i) {
    const int32_t page = a.block_table[(int64_t)request * a.max_blocks + odd[i].block];
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v_cache) +
                             ((int64_t)page * a.Hkv + head) * (int64_t)kBlock * a.d + col;
    for (int g = 0; g < 4; ++g)
      for (uint32_t m = odd[i].tokens[g]; m; m &= m - 1) {
        const int row = g * 32 + __ffs(m) - 1;
        if (!chunk_attends(pos, odd[i].block * kBlock + row, a.init, a.local)) continue;
        const float f = __bfloat162float(v[(int64_t)row * a.d]);
        if (!(fabsf(f) < INFINITY)) x += f;
      }
  }
  return x;
}

// Bits e < n of a word.
__device__ __forceinline__ uint32_t bits_below(int32_t n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Which of the tokens t0 .. t0 + 31 a row at `pos` attends.
__device__ __forceinline__ uint32_t attended_bits(int32_t pos, int32_t t0, int32_t init, int32_t local) {
  const int32_t from = local > pos ? 0 : pos - local + 1;  // its window's first token
  return bits_below(pos - t0 + 1) & (bits_below(init - t0) | ~bits_below(from - t0));
}

// Logits of hidden tokens to minus infinity.
__device__ __forceinline__ void hide(uint32_t* s, uint32_t on) {
  if (__all_sync(0xffffffffu, on == 0xffffffffu)) return;
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(on >> e & 1u)) s[e] = 0xff800000u;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Every lane holds N 16-byte pieces of its own row; after it, lane l holds piece l % N of rows N (l / N) + (k ^ l % N),
// k = 0 .. N - 1, of the warp, so that N lanes together hold a row's run of bytes.
template <int N>
__device__ __forceinline__ void transpose(uint32_t* v, int lane) {
#pragma unroll
  for (int b = 1; b < N; b <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (k & b) continue;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // piece k for the lane whose bit b is k's: each keeps one of its own and gets the other's like it
        uint32_t &x = v[4 * k + w], &y = v[4 * (k | b) + w];
        const uint32_t keep = lane & b ? y : x;
        y = __shfl_xor_sync(0xffffffffu, lane & b ? x : y, b);
        x = keep;
      }
    }
}

// While the plan is made: the pages that this CTA's first item is likely to begin with, into L2.  Only where all
// lists, each of a request of one tile, are cut into one round of parts.  This is ahead of the grid's wait, so what is
// read here may be older than the call: nothing but the choice of pages depends on it, each is checked to be one, and
// none of it stays in this SM's cache.  One token of 65536 52.3 -> 51.4 us, 4 over 16384 46.6 -> 44.8.
template <int D>
__device__ __forceinline__ void prefetch_first_pages(const ChunkArgs& a, int lane) {
  const int32_t lists = a.batch * a.Hkv, parts = a.ctas / lists;  // (lists <= ctas)
  const int32_t u = blockIdx.x % lists, part = blockIdx.x / lists;
  const int32_t r = (int32_t)a.by_heads.div(u), h = u - r * a.Hkv;
  const int32_t n = __ldcg(a.offsets + r + 1) - __ldcg(a.offsets + r);
  const int32_t L = (int32_t)min((int64_t)max(__ldcg(a.seq_lens + r), 0), (int64_t)a.max_blocks * kBlock);
  if (part >= parts || n <= 0 || n > a.tokens || n * a.G > kChunkTile) return;
  const ChunkPages g = chunk_pages(L - n, L - 1, a.init, a.local);
  const int32_t j = (int32_t)((int64_t)g.n * part / parts) + lane;
  if (lane >= kPrefetch || j >= g.n) return;
  const int32_t page = __ldcg(a.block_table + (int64_t)r * a.max_blocks + (j < g.na ? j : j + g.shift));
  if (page < 0 || (int64_t)page >= a.num_pages) return;
  const int64_t at = ((int64_t)page * a.Hkv + h) * Geo<D>::kTileBytes;
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char*>(a.k_cache) + at),
               "r"(Geo<D>::kTileBytes)
               : "memory");
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char*>(a.v_cache) + at),
               "r"(Geo<D>::kTileBytes)
               : "memory");
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_mma_kernel(const ChunkArgs a, const __grid_constant__ Maps maps) {
  using G = Geo<D>;
  extern __shared__ __align__(1024) unsigned char smem[];  // the swizzle's period
  auto& sh = *reinterpret_cast<Shared<G::kStages>*>(smem + G::kOffBar);
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 2);  // the products of both tiles
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_empty[i], 19);  // every warp but the one that takes items
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 2);
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&sh.v_part[i], 1);
      mbar_init(&sh.v_clean[i], 1);
    }
    mbar_init(&sh.turn[0], 1);
    mbar_init(&sh.turn[1], 1);
    mbar_init(&sh.drain[0], 1);
    mbar_init(&sh.drain[1], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      for (int c = 0; c < 2; ++c) mbar_init(&sh.p_full[i][c], 8);
      for (int w = 0; w < 4; ++w) mbar_init(&sh.pair[i][w], 2);
      mbar_init(&sh.o_full[i], 2);  // the products, and the notes of clean_values
    }
    fence_mbar_init();
    mbar_arrive(&sh.turn[0]);
  }
  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, 512);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = sh.tmem;
  if (warp == kPageWarp && (int64_t)a.batch * a.Hkv <= a.ctas) prefetch_first_pages<D>(a, lane);
  griddep_wait();
  griddep_launch_dependents();
  uint32_t eflags = 0;
  bool ok = true;  // no wait has run out
  Ring<kSlots> slot;
  // Next item for a consumer warp, in sh.item[slot.at] until done(): false at the end.
  auto take = [&] {
    ok = ok && mbar_wait(&sh.item_full[slot.at], slot.phase);
    return ok && sh.item[slot.at].request >= 0;
  };
  auto done = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.item_empty[slot.at]);
    slot.next();
  };

  if (warp >= kMmaWarp) {
    fewer_registers<kOtherRegs>();
    if (warp == kPageWarp) {
      // ---------------------------------------------------------------- items and pages
      ChunkHead* head = chunk_head(a);
      const int32_t n_items = head->items;
      const ChunkItem* items = reinterpret_cast<const ChunkItem*>(a.ws + a.lay.items);
      Ring<G::kStages> st;
      Ring<kParts> part;
      int64_t issued = 0;
      uint32_t info = 0;
      int32_t next = blockIdx.x;
      for (;;) {
        ok = ok && mbar_wait(&sh.item_empty[slot.at], slot.phase ^ 1);
        if (!ok) break;
        ChunkItem it;
        it.request = -1;
        if (next < n_items) it = items[next];
        if (lane == 0) {
          sh.item[slot.at] = it;
          sh.n_odd[slot.at] = 0;
          mbar_arrive(&sh.item_full[slot.at]);
        }
        slot.next();
        if (next >= n_items) break;
        int32_t p_lo, p_hi;
        item_span(it, a.by_group, p_lo, p_hi);
        for (int32_t j0 = it.j0; j0 < it.j1 && ok; j0 += 32) {
          int32_t page = 0, b = 0, seen = 0;
          if (j0 + lane < it.j1) {
            b = page_of(it, j0 + lane);
            page = a.block_table[(int64_t)it.request * a.max_blocks + b];
            if (chunk_masked(b, p_lo, p_hi, a.init, a.local)) seen = kPart;
            if (page < 0 || (int64_t)page >= a.num_pages) {
              eflags |= SRKV_EFLAG_PAGE_RANGE;
              page = (int32_t)a.num_pages;  // behind the cache: the copy fills with zeros
              seen |= kAbsent;
            }
          }
          const int n = min(32, it.j1 - j0);
          for (int i = 0; i < n && ok; ++i) {
            const int32_t z = __shfl_sync(0xffffffffu, page, i);
            const int32_t note = __shfl_sync(0xffffffffu, 4 * b + seen, i);
            for (int kv = 0; kv < 2 && ok; ++kv) {
              ok = mbar_wait(&sh.empty[st.at], st.phase ^ 1);
              if (!ok) break;
              if (lane == 0) {
                if (kv == 0) sh.page[info % kPageInfo] = note;
                unsigned char* dst = smem + G::kOffStage + (size_t)st.at * G::kTileBytes;
                mbar_arrive_expect_tx(&sh.full[st.at], G::kTileBytes);
#pragma unroll
                for (int b = 0; b < D / 64; ++b)
                  tma_page(dst + b * G::kBlockBytes, kv ? &maps.v : &maps.k, 64 * b, it.head * kBlock, z,
                           &sh.full[st.at]);
                if (kv == 1 && (note & kPart)) {
                  sh.part[part.at] = make_int2(st.at, (int)st.phase);
                  mbar_arrive(&sh.v_part[part.at]);
                }
              }
              __syncwarp();
              if (kv == 1 && (note & kPart)) part.next();
              st.next();
              ++issued;
            }
            ++info;
          }
        }
        if (lane == 0) next = atomicAdd(&head->next, 1) + (int32_t)gridDim.x;
        next = __shfl_sync(0xffffffffu, next, 0);
      }
      // every copy lands before the CTA ends: the last use of each stage
      for (int i = 0; i < G::kStages && i < issued; ++i) {
        if (st.at == 0) {
          st.at = G::kStages;
          st.phase ^= 1;
        }
        --st.at;
        ok = mbar_wait(&sh.full[st.at], st.phase) && ok;
      }
    } else if (warp < kPageWarp) {
      // ---------------------------------------------------------------- products
      constexpr uint32_t kQK = mma_desc(128, 128, false), kPV = mma_desc(128, D, true);
      const uint32_t q_desc = smem_desc(smem_u32(smem + G::kOffQ), 0);
      const uint32_t k_desc = smem_desc(smem_u32(smem + G::kOffStage), 0);
      const uint32_t v_desc = smem_desc(smem_u32(smem + G::kOffStage), G::kBlockBytes);
      Ring<G::kStages> st;
      const int i = warp - kMmaWarp;  // the tile
      Ring<1> qr, pr, tr;
      Ring<kParts> part;
      uint32_t info = 0;
      // S_i = Q_i K^T; before the last steps the other tile's warp is told (where both are in use), so that its first
      // product is there when these are through.
      auto qk = [&](int s, bool tell) {
        const uint32_t q = q_desc + i * (G::kTileBytes >> 4), k = k_desc + s * (G::kTileBytes >> 4);
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          const uint32_t off = ((e / 4) * G::kBlockBytes + (e % 4) * 32) >> 4;
          if (e == D / 16 - kTellAhead && tell) mbar_arrive(&sh.turn[i ^ 1]);
          mma_ss(tmem + G::kS + 128 * i, q + off, k + off, kQK, e > 0);
        }
        mma_commit(&sh.s_full[i]);
      };
      // O_i (+)= P_i V over a part of the tokens; each half of P lies at the start of its half of S.
      auto pv = [&](int s, int c, bool first) {
        const uint32_t v = v_desc + s * (G::kTileBytes >> 4);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mma_ts(tmem + G::kO + D * i, tmem + G::kS + 128 * i + 64 * h + 8 * (2 * c + e),
                   v + (4 * h + 2 * c + e) * (2048 >> 4), kPV, !first || c + h + e > 0);
      };
      while (take()) {
        const ChunkItem& it = sh.item[slot.at];
        const int32_t n = it.j1 - it.j0;
        const bool alone = it.rows <= 128;  // tile 1 is not in use: tile 0's warp lets go of the stages for both
        if (n > 0) {
          ok = ok && mbar_wait(&sh.q_full, qr.phase);
          if (!ok) break;
          qr.next();
        }
        if (alone && i == 1) {
          if (n > 0 && lane == 0) mbar_arrive(&sh.q_empty);
          int32_t p_lo, p_hi;
          item_span(it, a.by_group, p_lo, p_hi);
          for (int32_t j0 = it.j0; j0 < it.j1; j0 += 32)
            part.skip(__popc(__ballot_sync(
                0xffffffffu, j0 + lane < it.j1 &&
                                 chunk_masked(page_of(it, j0 + lane), p_lo, p_hi, a.init, a.local))));
          st.skip(2 * n);
          info += n;
          done();
          continue;
        }
        auto release = [&](uint64_t* bar) {
          mma_commit(bar);
          if (alone) mma_commit(bar);
        };
        // The tiles' blocks of products alternate: in step, one's run while the other is at its exponentials.
        auto my_turn = [&] {
          if (!alone) {
            ok = ok && mbar_wait(&sh.turn[i], tr.phase);
            tr.next();
          }
          return ok;
        };
        if (n > 0) {
          ok = mbar_wait(&sh.full[st.at], st.phase);
          if (!ok || !my_turn()) break;
          tcgen05_fence_after();
          if (lane == 0) {
            qk(st.at, !alone);
            release(&sh.empty[st.at]);
            if (n == 1) mma_commit(&sh.q_empty);
          }
          __syncwarp();
        }
        for (int32_t j = 0; j < n && ok; ++j, st = st.plus(2)) {
          const Ring<G::kStages> v = st.plus(1), k = st.plus(2);
          const bool more = j + 1 < n;
          ok = mbar_wait(&sh.full[v.at], v.phase) && (!more || mbar_wait(&sh.full[k.at], k.phase));
          if (!ok) break;
          if (sh.page[info++ % kPageInfo] & kPart) {
            ok = mbar_wait(&sh.v_clean[part.at], part.phase);
            if (!ok) break;
            part.next();
          }
          for (int c = 0; c < 2 && ok; ++c) {
            ok = mbar_wait(&sh.p_full[i][c], pr.phase);
            if (!ok || (c == 0 && !my_turn())) break;
            tcgen05_fence_after();
            if (lane == 0) pv(v.at, c, j == 0);
            __syncwarp();
          }
          if (!ok) break;
          pr.next();
          if (lane == 0) {
            if (more) {
              qk(k.at, !alone);
              release(&sh.empty[v.at]);
              release(&sh.empty[k.at]);
              if (j + 2 == n) mma_commit(&sh.q_empty);
            } else {
              mma_commit(&sh.o_full[i]);
              if (!alone) mbar_arrive(&sh.turn[i ^ 1]);
              mbar_arrive(&sh.o_full[i]);
              release(&sh.empty[v.at]);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        done();
      }
      if (!ok) {  // a wait ran out: products in flight still end before the tensor memory is freed
        if (lane == 0) mma_commit(&sh.drain[i]);
        __syncwarp();
        mbar_wait(&sh.drain[i], 0);
      }
    } else {
      // ---------------------------------------------------------------- queries, and values to be cleaned
      Ring<kParts> part;
      Ring<1> qr;
      while (take()) {
        const ChunkItem& it = sh.item[slot.at];
        if (it.j1 > it.j0) {
          ok = ok && mbar_wait(&sh.q_empty, qr.phase ^ 1);
          if (!ok) break;
          qr.next();
          if (maps.q_box > 0) {  // a tile's tokens and heads are a box, its rows in their order
            if (lane == 0) {
              const int tiles = it.rows > 128 ? 2 : 1;
              mbar_arrive_expect_tx(&sh.q_full, tiles * G::kTileBytes);
              for (int i = 0; i < tiles; ++i)
#pragma unroll
                for (int b = 0; b < D / 64; ++b)
                  tma_page(smem + G::kOffQ + i * G::kTileBytes + b * G::kBlockBytes, &maps.q, 64 * b,
                           it.head * a.G, it.tok0 + (int32_t)a.by_group.div(it.row0) + i * maps.q_box, &sh.q_full);
            }
          } else {
            constexpr int C = D / 8, kStep = 32 / C;  // 16-byte chunks of a row, rows a pass
            const int t = lane, chunk = t % C;
            const int32_t rho = it.row0 + t / C, head0 = it.head * a.G;
            int32_t token = (int32_t)a.by_group.div(rho), g = rho - token * a.G;
            const int32_t dt = (int32_t)a.by_group.div(kStep), dg = kStep - dt * a.G;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)it.tok0 * a.q_stride + chunk * 8;
            const int32_t rows = it.rows;
#pragma unroll 4
            for (int row = t / C; row < rows; row += kStep) {
              const uint32_t dst = smem_u32(smem + G::kOffQ) + (row / 128) * G::kTileBytes +
                                   (chunk / 8) * G::kBlockBytes + (row % 128) * 128 + ((chunk ^ row) % 8) * 16;
              cp_async_16(dst, q + (int64_t)token * a.q_stride + (head0 + g) * D);
              token += dt;
              g += dg;
              if (g >= a.G) {
                g -= a.G;
                ++token;
              }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0 && maps.q_box == 0) mbar_arrive(&sh.q_full);
        }
        // the values of pages seen in part, ahead of their product
        int32_t p_lo, p_hi;
        item_span(it, a.by_group, p_lo, p_hi);
        for (int32_t j = it.j0; j < it.j1 && ok; ++j) {
          const int32_t b = page_of(it, j);
          if (!chunk_masked(b, p_lo, p_hi, a.init, a.local)) continue;
          ok = mbar_wait(&sh.v_part[part.at], part.phase);
          if (!ok) break;
          const int2 where = sh.part[part.at];
          ok = mbar_wait(&sh.full[where.x], (uint32_t)where.y);
          if (!ok) break;
          bool wrote = false;
          const int n_odd = sh.n_odd[slot.at];
          uint32_t any = 0;
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            const int32_t t = b * kBlock + 32 * g + lane;
            const bool behind = t >= it.L;
            // a token that the first row and the last one see is seen by all between; by neither, by none
            const bool scan = !behind && !(chunk_attends(p_lo, t, a.init, a.local) &&
                                           chunk_attends(p_hi, t, a.init, a.local));
            const uint32_t bad = clean_values<D>(
                smem + G::kOffStage + (size_t)where.x * G::kTileBytes + g * (32 * 128), behind, scan, lane);
            wrote |= bad || __any_sync(0xffffffffu, behind);
            any |= bad;
            if (lane == 0 && n_odd < kOdd) sh.odd[slot.at][n_odd].tokens[g] = bad;
          }
          if (lane == 0 && any && n_odd < kOdd) {
            sh.odd[slot.at][n_odd].block = b;
            sh.n_odd[slot.at] = n_odd + 1;
          }
          if (wrote) fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.v_clean[part.at]);
          part.next();
        }
        done();
      }
      if (!ok) mbar_wait(&sh.q_full, qr.phase ^ 1);  // a wait ran out: a copy in flight lands before the CTA ends
    }
  } else {
    more_registers<kSoftmaxRegs>();
    // ---------------------------------------------------------------- softmax and output
    const int tile = warp / 8, half = warp / 4 % 2, quad = warp % 4, in_tile = 32 * quad + lane;
    const int row = 128 * tile + in_tile;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t ts = tmem + G::kS + 128 * tile + 64 * half + lanes;
    const uint32_t to = tmem + G::kO + D * tile + D / 2 * half + lanes;
    const float scale = a.scale_log2;
    Ring<1> sr, orr, xr;
    // Both warps of a row wait for each other's note in shared memory.
    auto exchange = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.pair[tile][quad]);
      ok = mbar_wait(&sh.pair[tile][quad], xr.phase);
      xr.next();
    };
    uint32_t info = 0;
    while (take()) {
      const ChunkItem& it = sh.item[slot.at];
      const int32_t n = it.j1 - it.j0;
      const bool here = 128 * tile < it.rows;              // the tile is in use
      const bool work = 128 * tile + 32 * quad < it.rows;  // some row of this warp is
      const bool mine = row < it.rows;                     // this lane's row is
      const int32_t pos = it.p0 + (int32_t)a.by_group.div(it.row0 + row);
      const float most = it.rows <= 128 ? 0.f : kGrow;
      float m = -INFINITY;
      float2 sum = make_float2(0.f, 0.f);
      for (int32_t j = 0; here && j < n && ok; ++j, ++info) {
        ok = mbar_wait(&sh.s_full[tile], sr.phase);
        if (!ok) break;
        sr.next();
        tcgen05_fence_after();
        if (work) {
          uint32_t s[64];
          tmem_ld32(ts, s);
          tmem_ld32(ts + 32, s + 32);
          const int32_t page = sh.page[info % kPageInfo];
          tmem_wait_ld();
          tmem_use32(s);
          tmem_use32(s + 32);
          uint32_t late = 0xffffffffu;  // what the row attends of the second 32 tokens
          if (page & 3) {
            const int32_t t0 = (page >> 2) * kBlock + 64 * half;
            hide(s, !(page & kAbsent) ? attended_bits(pos, t0, a.init, a.local) : 0u);
            late = !(page & kAbsent) ? attended_bits(pos, t0 + 32, a.init, a.local) : 0u;
            hide(s + 32, late);
          }
          float top[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 4]));
#pragma unroll
          for (int e = 8; e < 64; e += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top[i] = max3(top[i], __uint_as_float(s[e + i]), __uint_as_float(s[e + i + 4]));
          const float here_top = max3(fmaxf(top[0], top[1]), top[2], top[3]);
          sh.note[tile][half][in_tile] = here_top;  // read before this page's P is complete, so before the next S
          exchange();
          if (!ok) break;
          const float now = max3(m, here_top, sh.note[tile][half ^ 1][in_tile]);
          if (j == 0) {
            m = now;
          } else {
            const bool grow = mine && (now - m) * scale > most;
            if (__any_sync(0xffffffffu, grow)) {
              const float w = grow ? fast_exp2((m - now) * scale) : 1.f;
              if (grow) m = now;
              sum.x *= w;
              sum.y *= w;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[16];
                tmem_ld16(to + 16 * c, o);
                tmem_wait_ld();
                tmem_use16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * w);
                tmem_st16(to + 16 * c, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : -m * scale;
          const float2 scale2 = make_float2(scale, scale), ref2 = make_float2(ref, ref);
          float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          // the second half of the logits is read again rather than held over all this
          tmem_ld32(ts + 32, s + 32);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c == 1) {
              tmem_wait_ld();
              tmem_use32(s + 32);
              if (page & 3) hide(s + 32, late);
            }
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float2 x = __ffma2_rn(
                  make_float2(__uint_as_float(s[32 * c + e]), __uint_as_float(s[32 * c + e + 1])), scale2, ref2);
              x.x = fast_exp2(x.x);
              x.y = fast_exp2(x.y);
              part[(e / 2) % 2] = __fadd2_rn(part[(e / 2) % 2], x);
              p[e / 2] = pack_bf16(x.x, x.y);
            }
            tmem_st16(ts + 16 * c, p);
            tmem_wait_st();
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[tile][c]);
          }
          sum = __fadd2_rn(sum, __fadd2_rn(part[0], part[1]));
        } else if (lane == 0) {
          mbar_arrive(&sh.p_full[tile][0]);
          mbar_arrive(&sh.p_full[tile][1]);
        }
      }
      if (!here) info += n;
      if (!ok) break;
      if (here) {
        float l = 0.f;
        if (n > 0) {
          ok = mbar_wait(&sh.o_full[tile], orr.phase);
          if (!ok) break;
          orr.next();
          tcgen05_fence_after();
          if (work) {
            l = sum.x + sum.y;
            sh.note[tile][half][in_tile] = l;
            exchange();
            if (!ok) break;
            const float other = sh.note[tile][half ^ 1][in_tile];
            l = half ? other + l : l + other;
            exchange();  // before the next item's notes
            if (!ok) break;
          }
        }
        if (work) {
          const int n_odd = n > 0 ? sh.n_odd[slot.at] : 0;
          const int32_t rho = it.row0 + row;
          // A row without a finite logit is zero whatever its values are; a partial result of one keeps what it has, as
          // another part may have a weight.
          const bool none = l == 0.f && it.slot < 0, some = __any_sync(0xffffffffu, none);
          const float w = it.slot >= 0 ? 1.f : 1.f / l;
          const int col = D / 2 * half;
          // rows of the output that this warp's lanes stand for, -1: none
          const int32_t token = (int32_t)a.by_group.div(rho);
          const int32_t at = !mine ? -1
                             : it.slot >= 0 ? it.slot + row
                                            : (it.tok0 + token) * a.Hq + it.head * a.G + (rho - token * a.G);
          const float2 w2 = make_float2(w, w);
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            if (n > 0) {
              tmem_ld32(to + 32 * c, o);
              tmem_wait_ld();
              tmem_use32(o);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 x = __fmul2_rn(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), w2);
                o[e] = __float_as_uint(x.x);
                o[e + 1] = __float_as_uint(x.y);
              }
              if (some) {  // (a branch that next to no warp takes: 64 selects took 1 % of 1024 single tokens over 512)
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = none ? 0u : o[e];
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0;
            }
            if (n_odd > 0 && mine && !none) {
#pragma unroll 1
              for (int e = 0; e < 32; ++e) {
                const float x =
                    odd_value(a, it.request, it.head, sh.odd[slot.at], n_odd, pos, col + 32 * c + e);
#pragma unroll
                for (int f = 0; f < 32; ++f)
                  if (f == e) o[f] = __float_as_uint(__uint_as_float(o[f]) + x);
              }
            }
            if (it.slot >= 0) {
              transpose<8>(o, lane);
              float* acc = reinterpret_cast<float*>(a.ws + a.lay.acc) + col + 32 * c + 4 * (lane % 8);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int32_t r = __shfl_xor_sync(0xffffffffu, at, k);
                if (r >= 0)
                  *reinterpret_cast<uint4*>(acc + (int64_t)r * D) =
                      make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
              }
            } else {
              uint32_t v[16];
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                v[e / 2] = pack_bf16(__uint_as_float(o[e]), __uint_as_float(o[e + 1]));
              transpose<4>(v, lane);
              __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + col + 32 * c + 8 * (lane % 4);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int32_t r = __shfl_xor_sync(0xffffffffu, at, k);
                if (r >= 0)
                  *reinterpret_cast<uint4*>(out + (int64_t)r * D) =
                      make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
              }
            }
          }
          if (mine && half == 0 && it.slot >= 0)
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.ws + a.lay.ml) + 2 * (int64_t)(it.slot + row)) =
                make_float2(m == -INFINITY ? m : m * scale, l);
        }
        tcgen05_fence_before();
      }
      done();
    }
  }
  if (!ok) eflags |= SRKV_EFLAG_TIMEOUT;
  eflags = __reduce_or_sync(0xffffffffu, eflags);
  if (lane == 0) raise_flags(a.error_flags, eflags);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 512);
}

template <int D>
cudaError_t launch_d(const ChunkArgs& a, cudaStream_t stream) {
  using G = Geo<D>;
  constexpr size_t smem = G::kOffBar + sizeof(Shared<G::kStages>);
  static_assert(smem <= 232448, "shared memory opt-in limit");
  static_assert(G::kStages <= 2 * kParts && G::kStages <= 8, "rings");
  // The shared-memory opt-in is set once per device (not during graph capture).
  static bool configured[128] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(chunk_mma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  Maps maps;
  if (!encode_cache_map(&maps.k, a.k_cache, a.num_pages, a.Hkv, D, false) ||
      !encode_cache_map(&maps.v, a.v_cache, a.num_pages, a.Hkv, D, false))
    return cudaErrorInvalidValue;
  maps.q_box = a.G <= 128 && 128 % a.G == 0 ? 128 / a.G : 0;
  if (maps.q_box > 0 &&
      !encode_rows_map(&maps.q, a.q, a.tokens, a.q_stride, a.Hq, D, a.G, maps.q_box))
    return cudaErrorInvalidValue;
  return launch_pdl(chunk_mma_kernel<D>, dim3(a.ctas), dim3(kThreads), smem, stream, a, maps);
}

}  // namespace

cudaError_t launch_chunk_mma(const ChunkArgs& a, cudaStream_t stream) {
  return a.d == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace srkv
