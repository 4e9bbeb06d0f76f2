// chunk_plan.cuh -- how the attention of a chunk of new tokens is divided: shared by the plan kernel, the two
// attention kernels and the merge.
//
// The rows of one (request, kv head) are its new tokens' query heads, row = token * G + head of the group, so
// that one read of a page serves all of them whatever G is.  They are cut into tiles of kChunkTile rows (on
// CUDA cores of 64 or 128).  A tile attends a list of pages in ascending order: those below `na`, then, with a
// window, those from page na + shift on.  A long list may be divided among several items; their partial results are
// merged (chunk_plan.cu).
#pragma once

#include "srkv_internal.cuh"

namespace srkv {

constexpr int kChunkTile = 256;      // rows of a tile on tensor cores: two accumulators of 128
constexpr int kChunkTileSimt64 = 64, kChunkTileSimt128 = 128;  // rows of a tile on CUDA cores, by head size
constexpr int32_t kChunkSplitItems = 4096;    // items that divided lists may add
constexpr int32_t kChunkPartRows = 163840;    // rows of partial results: 640 tiles of 256
constexpr int32_t kChunkPartsPerRow = 512;    // and no more than this many for every row

// One unit of work: rows [row0, row0 + rows) of (request, head) over positions [j0, j1) of the tile's page list.
struct __align__(16) ChunkItem {
  int32_t request, head;
  int32_t row0, rows;
  int32_t j0, j1;
  int32_t na, shift;  // position j is page j below na, else page j + shift
  int32_t slot;       // first row of its partial result, or -1: the tile's output is this item's
  int32_t tok0;       // row of the packed inputs where the request's chunk starts
  int32_t p0;         // position of that token (negative where the chunk is longer than its sequence)
  int32_t L;          // the request's length
};
static_assert(sizeof(ChunkItem) == 48, "three 16-byte loads");

// A tile whose list was divided: `parts` partial results of `rows` rows each, one behind the other from `slot`.
struct __align__(16) ChunkMerge {
  int32_t head, row0, rows, tok0;
  int32_t slot, parts;
};
static_assert(sizeof(ChunkMerge) == 32, "two loads");

// Division of any 32-bit number by one known on the host, as a multiplication (Granlund and Montgomery, "Division by
// Invariant Integers using Multiplication", 1994, figure 4.1).
struct DivideBy {
  uint32_t m, s1, s2;
  static DivideBy of(uint32_t d) {
    uint32_t l = 0;
    while (l < 32 && (1ull << l) < d) ++l;
    return {(uint32_t)((((1ull << l) - d) << 32) / d + 1), l < 1 ? l : 1, l > 0 ? l - 1 : 0};
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    const uint32_t t = __umulhi(m, n);
    return (t + ((n - t) >> s1)) >> s2;
  }
};

struct ChunkHead {  // counters of one call, written by the plan (read word by word in the merge)
  int32_t items, merges;  // merges: divided tiles times heads
  int32_t next;       // the next item to hand out
  int32_t merge_rows, merge_parts;  // rows, and parts, of the largest merge
};

// Workspace (256-byte aligned parts).
struct ChunkLayout {
  size_t req;      // int32[2 * batch + 2]: first tile of each request, tokens of each request (0: none or refused)
  size_t items;    // ChunkItem[items_cap]
  size_t merges;   // ChunkMerge[merges_cap]
  size_t ml;       // float[rows_cap][2]: maximum (log2 domain) and sum
  size_t acc;      // float[rows_cap][d]: unnormalised outputs
  size_t total;
  int32_t items_cap, merges_cap, rows_cap;
};

struct ChunkArgs {
  const void* q;
  int64_t q_stride;  // elements between tokens
  const void* k_cache;
  const void* v_cache;
  int64_t num_pages;
  const int32_t* block_table;
  int32_t max_blocks;
  const int32_t* offsets;
  int32_t tokens;
  const int32_t* seq_lens;
  int32_t batch;
  void* out;
  char* ws;
  ChunkLayout lay;
  int32_t* error_flags;
  int32_t Hq, Hkv, G, d;
  int32_t init, local;  // without a window: init = INT32_MAX, local = 0
  float scale_log2;     // log2(e) / sqrt(d)
  int32_t tile_log2;    // rows of a tile
  int32_t ctas;         // CTAs that take items
  float per_cta;        // 1 / ctas
  float page_rate;      // how fast a page is, of the tensor cores' rate
  DivideBy by_group, by_heads;  // by G and Hkv
};

__host__ __device__ __forceinline__ ChunkHead* chunk_head(const ChunkArgs& a) {
  return reinterpret_cast<ChunkHead*>(a.ws);
}

// The page list of a tile whose rows stand at positions p_lo .. p_hi.
struct ChunkPages {
  int32_t na, shift, n;
};
__host__ __device__ __forceinline__ ChunkPages chunk_pages(int32_t p_lo, int32_t p_hi, int32_t init,
                                                           int32_t local) {
  ChunkPages g = {0, 0, 0};
  if (p_hi < 0) return g;
  const int32_t first = init < p_hi + 1 ? init : p_hi + 1;
  g.na = first / kBlock + (first % kBlock != 0);
  g.n = g.na;
  if (local > 0) {
    const int32_t from = p_lo + 1 > local ? p_lo + 1 - local : 0;
    const int32_t b0 = from / kBlock > g.na ? from / kBlock : g.na;
    const int32_t b1 = p_hi / kBlock + 1;
    g.shift = b0 - g.na;
    if (b1 > b0) g.n += b1 - b0;
  }
  return g;
}

// Does a row at position p attend token t?
__device__ __forceinline__ bool chunk_attends(int32_t p, int32_t t, int32_t init, int32_t local) {
  return t <= p && (t < init || p - t < local);
}

// Is some token of page b hidden from some row at positions p_lo .. p_hi?
__device__ __forceinline__ bool chunk_masked(int32_t b, int32_t p_lo, int32_t p_hi, int32_t init,
                                             int32_t local) {
  const int32_t t0 = b * kBlock, t1 = t0 + kBlock - 1;
  return t1 > p_lo || (t1 >= init && t0 <= p_hi - local);
}

// Rows of a tile under a configuration.
int32_t chunk_tile(const srkv_config& cfg);
size_t chunk_workspace(const srkv_config& cfg, int32_t tokens, int32_t batch, ChunkLayout* lay);
cudaError_t launch_chunk_plan(const ChunkArgs& a, cudaStream_t stream);
cudaError_t launch_chunk_merge(const ChunkArgs& a, int32_t dtype, cudaStream_t stream);
cudaError_t launch_chunk_simt(const ChunkArgs& a, cudaStream_t stream);
cudaError_t launch_chunk_mma(const ChunkArgs& a, cudaStream_t stream);

}  // namespace srkv
