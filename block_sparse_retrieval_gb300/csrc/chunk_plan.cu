// chunk_plan.cu -- the plan of a chunk's attention, and the merge of divided lists.
//
// Lengths live on the device, so the work is divided there: one CTA lists the items, longest first, and the
// attention kernel's CTAs take them one by one.  Lists are kept whole where they balance by themselves; else they are
// cut: where they are fewer than CTAs all of them, else those that remain after full rounds of whole ones; where they are
// many (16 and more a CTA, or of more tiles than are held on chip), those longer than the average load, each by its own
// length.
//
// This kernel's time is the fetch of its own instructions (a launch finds none of them on its SM: some 300 cycles
// for every 8), not its arithmetic.  So loops are kept rolled, divisions by the head counts are multiplications, and
// what is done twice is a function: 16.4 us with the loops unrolled, some 6 so (one request).
#include "chunk_plan.cuh"

namespace srkv {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kBuckets = 64;   // sizes 0 .. 3, then two per octave
constexpr int kHeld = 512;     // requests, and tiles, that are held on chip
// What starting and ending an item costs, what the merge adds, and each row of a partial result, in pages on tensor
// cores (1.6 us); a page on CUDA cores takes ten times that.  One figure each for both head sizes and for items of all
// sizes, whose pages differ by 2 and more: whether and where lists are cut hangs on them, no result's bounds do.
constexpr float kItemCost = 2.f, kMergeCost = 2.f, kRowCost = 1.f / 8192;

__device__ __forceinline__ int bucket_of(int32_t n) {
  if (n < 4) return n;
  const int e = 31 - __clz(n);
  return 2 * e + ((n >> (e - 1)) & 1);
}

// How lists are cut: those of the first `whole` tiles not at all; the others, one behind the other (tile by tile,
// head by head), at every `grid` pages, or, if `parts` > 0, each into that many equal parts, or, if `most` > 0, each
// into as few equal parts as are no longer than that.
struct Cuts {
  int32_t whole, grid, parts, most;
};

// The requests as the plan sees them: on chip while they are few, else in the workspace and the call's arrays.
struct Requests {
  const int32_t* first;  // first tile of each
  const int32_t* n;      // its new tokens (0: none, or refused)
  const int32_t* offset;
  const int32_t* len;
  int32_t count;
};

struct Tile {
  int32_t request, row0, rows, tok0, p0, L;
  ChunkPages g;
};

__device__ __noinline__ Tile load_tile(const ChunkArgs& a, const Requests& q, int32_t tau) {
  Tile t;
  int32_t lo = 0, hi = q.count;  // the last request whose first tile is at or before tau
#pragma unroll 1
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (q.first[mid] <= tau)
      lo = mid;
    else
      hi = mid;
  }
  t.request = lo;
  const int32_t n = q.n[lo];
  t.row0 = (tau - q.first[lo]) << a.tile_log2;
  t.rows = min(1 << a.tile_log2, n * a.G - t.row0);
  t.tok0 = q.offset[lo];
  t.L = (int32_t)min((int64_t)max(q.len[lo], 0), (int64_t)a.max_blocks * kBlock);
  t.p0 = t.L - n;
  t.g = chunk_pages(t.p0 + (int32_t)a.by_group.div(t.row0), t.p0 + (int32_t)a.by_group.div(t.row0 + t.rows - 1),
                    a.init, a.local);
  return t;
}

// The pieces of list h of a tile: the first one's end, the length of the next ones, and how many there are.
struct Pieces {
  int32_t first, each, count;
};
__device__ __noinline__ Pieces pieces_of(const Cuts& cut, int32_t t, int32_t h, int32_t n, long long before,
                                         int32_t heads) {
  Pieces p = {n, 1, 1};
  if (t >= cut.whole) {
    p.each = cut.grid;
    if (cut.parts > 0 || cut.most > 0) {
      const int32_t parts = cut.parts > 0 ? cut.parts : max(1, (n + cut.most - 1) / cut.most);
      p.each = max(1, (n + parts - 1) / parts);
      p.first = min(n, p.each);
    } else {
      // the row of lists is cut where its position is a multiple of the grid (rows of 2^32 pages are not cut)
      p.first = min(n, cut.grid - (int32_t)((uint32_t)(before * heads + (long long)h * n) % (uint32_t)cut.grid));
    }
    p.count = 1 + (n - p.first + p.each - 1) / p.each;
  }
  return p;
}

template <typename I>
__device__ __forceinline__ I warp_scan(I v, int lane) {
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const I y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Inclusive sum over the CTA's threads; *all is the whole sum.  `sums`: a word for each warp.
__device__ __noinline__ long long block_scan(long long v, long long* sums, long long* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  const long long w = warp_scan(lane < kPlanWarps ? sums[lane] : 0ll, lane);
  *all = __shfl_sync(0xffffffffu, w, kPlanWarps - 1);
  if (warp > 0) v += __shfl_sync(0xffffffffu, w, warp - 1);
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ int32_t hist[kBuckets];
  __shared__ int32_t held[4][kHeld];
  __shared__ Tile tile[kHeld];
  __shared__ long long before[kHeld];  // pages of the tiles before, for one head
  __shared__ long long sums[kPlanWarps];
  __shared__ int32_t n_items, n_placed, n_merges, n_rows, max_parts, longest, shortest, most_rows;
  __shared__ Cuts cut;
  __shared__ bool equal;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kBuckets) hist[tid] = 0;
  if (tid == 0) {
    n_items = n_placed = n_merges = n_rows = max_parts = longest = most_rows = 0;
    shortest = INT32_MAX;
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the requests' tiles
  const bool few = a.batch <= kHeld;
  int32_t* req = reinterpret_cast<int32_t*>(a.ws + a.lay.req);
  uint32_t eflags = 0;
  // tiles that good offsets make at most
  const int32_t cap = a.lay.items_cap / a.Hkv - (kChunkSplitItems + a.Hkv - 1) / a.Hkv;
  long long base = 0;
#pragma unroll 1
  for (int32_t r0 = 0; r0 < a.batch; r0 += kPlanThreads) {
    const int32_t r = r0 + tid;
    int32_t n = 0, s = 0, len = 0;
    if (r < a.batch) {
      s = a.offsets[r];
      const int32_t e = a.offsets[r + 1];
      len = a.seq_lens[r];
      if (s < 0 || e < s || e > a.tokens)
        eflags |= SRKV_EFLAG_CHUNK;
      else
        n = e - s;
      if (n > 0) {
        if (len < 0 || (int64_t)len > (int64_t)a.max_blocks * kBlock) eflags |= SRKV_EFLAG_SEQ_LEN;
        if (n > len) eflags |= SRKV_EFLAG_CHUNK;
      }
    }
    const long long mine = ((int64_t)n * a.G + (1 << a.tile_log2) - 1) >> a.tile_log2;
    long long all;
    const long long upto = base + block_scan(mine, sums, &all);
    if (r < a.batch) {
      // offsets that go back and forth could ask for more tiles than the workspace holds
      if (upto > cap) eflags |= SRKV_EFLAG_CHUNK;
      const int32_t first = (int32_t)min(upto - mine, (long long)cap);
      if (few) {
        held[0][tid] = first;
        held[1][tid] = n;
        held[2][tid] = s;
        held[3][tid] = len;
      } else {
        req[r] = first;
        req[a.batch + 1 + r] = n;
      }
    }
    base = min(base + all, (long long)cap);
  }
  __syncthreads();
  const int32_t tiles = (int32_t)base;
  const Requests q = {few ? held[0] : req, few ? held[1] : req + a.batch + 1, few ? held[2] : a.offsets,
                      few ? held[3] : a.seq_lens, a.batch};

  // ---- their page lists, and the pages before each
  long long pages = 0;
#pragma unroll 1
  for (int32_t t0 = 0; t0 < tiles; t0 += kPlanThreads) {
    const int32_t t = t0 + tid;
    int32_t n = 0;
    if (t < tiles) {
      const Tile tl = load_tile(a, q, t);
      n = tl.g.n;
      atomicMax(&longest, n);
      atomicMin(&shortest, n);
      atomicMax(&most_rows, tl.rows);
      if (t < kHeld) tile[t] = tl;
    }
    long long all;
    const long long upto = pages + block_scan(n, sums, &all);
    if (t < kHeld) before[t] = upto - n;
    pages += all;
  }
  __syncthreads();

  // ---- whole lists, or cut ones
  const int32_t lists = tiles * a.Hkv;
  if (tid == 0) {
    Cuts c = {tiles, 1, 0, 0};
    // whole lists: the average load; or the longest one; or, with some CTAs idle while the last lists run, the
    // load and those CTAs' share of a shortest list
    const float load = (float)pages * (float)a.Hkv * a.per_cta;
    const float items = (float)lists * a.per_cta, idle = ceilf(items) - items;
    const float item = kItemCost * a.page_rate, merge = kMergeCost * a.page_rate;
    const float whole = fmaxf((float)longest, load + idle * (float)shortest) + item * ceilf(items);
    if (tiles <= kHeld && lists < 16 * a.ctas) {
      // Full rounds of whole lists, and the rest cut; else all cut, where one list is longer than the average load, too
      // (4 ragged chunks of up to 600 over 32768 tokens 243 -> 136 us).
      const bool many = lists >= a.ctas, rounds = many && (float)longest <= load;
      c.whole = rounds ? (int32_t)a.by_heads.div((int32_t)items * a.ctas) : 0;
      const float rest =
          rounds ? (float)(c.whole < tiles ? pages - before[c.whole] : 0) * (float)a.Hkv * a.per_cta : load;
      // One piece for each CTA, or two (after rounds; on CUDA cores, whose pages take longer than a piece's start and
      // end, from 8 pages on: 7 ragged chunks of 9 pages a CTA 175 -> 169 us, 3 of 3 pages 65 -> 72).
      const int32_t cut_lists = lists - c.whole * a.Hkv;
      // Partial results are those of the lists that are cut: no more of them than there are cuts (one more than planned,
      // as the average load is rounded), and a piece more than cuts each.
      auto fits = [&](int32_t cuts) {
        const int32_t partial = cuts + min(cuts, cut_lists);
        return partial <= kChunkSplitItems && (int64_t)partial * most_rows <= a.lay.rows_cap;
      };
      int32_t k = rounds || (a.page_rate < 1.f && rest >= 8.f) ? 2 : 1;
      if (!fits(k * a.ctas + 1)) k = 1;  // a tile or two of one head on CUDA cores
      const int32_t pieces = cut_lists + k * a.ctas;
      c.grid = max(a.page_rate < 1.f ? 1 : 2, (int32_t)ceilf(fminf(rest / (float)k, 1e9f)));
      float cost = load + item * (many ? items + 2.f : 2.f) + merge;
      if (!rounds && longest == shortest) {  // equal lists: into as many equal parts as make one round
        const int32_t parts = (int32_t)((float)a.ctas / (float)max(lists, 1));
        const float each = ceilf((float)longest / (float)parts) + item + merge;
        if (parts > 1 && each <= cost) {
          cost = each;
          c.parts = parts;
        }
      }
      cost += (float)pieces * (float)most_rows * kRowCost * a.page_rate;
      if (cost >= whole || !fits(k * a.ctas + 1) || pages * a.Hkv > (long long)UINT32_MAX)
        c = {tiles, 1, 0, 0};
    } else if ((float)longest > load) {
      // A list of n > most pages has fewer than 2 n / most parts, so all have fewer than 2 load / most a CTA, whose
      // partial results have to fit (and some to spare for the rounding of the load).
      const float most = ceilf(1.001f * load * fmaxf(1.f, 2.f * (float)a.ctas * (float)most_rows / (float)a.lay.rows_cap));
      const float cost = load + item * (ceilf(items) + 2.f) + merge +
                         2.f * (float)a.ctas * (float)most_rows * kRowCost * a.page_rate;
      if (cost < whole && most < (float)longest) c = {0, 1, 0, (int32_t)most};
    }
    cut = c;
    equal = longest == shortest && (c.whole == tiles || c.parts > 0);
  }
  __syncthreads();

  // ---- the longest items come first, unless all are as good as equal: the sizes, and from them the places
  if (!equal) {
#pragma unroll 1
    for (int32_t u = tid; u < lists; u += kPlanThreads) {
      const int32_t t = (int32_t)a.by_heads.div(u), h = u - t * a.Hkv;
      const int32_t n = t < kHeld ? tile[t].g.n : load_tile(a, q, t).g.n;
      const Pieces p = pieces_of(cut, t, h, n, t < kHeld ? before[t] : 0, a.Hkv);
      atomicAdd(&hist[bucket_of(p.first)], 1);
      if (p.count > 1) {
        atomicAdd(&hist[bucket_of(n - p.first - (p.count - 2) * p.each)], 1);
        if (p.count > 2) atomicAdd(&hist[bucket_of(p.each)], p.count - 2);
      }
    }
    __syncthreads();
    if (warp == 0) {
      int32_t at = 0;
#pragma unroll 1
      for (int b = kBuckets - 1 - lane; b >= 0; b -= 32) {
        const int32_t n = hist[b], upto = at + warp_scan(n, lane);
        hist[b] = upto - n;
        at = __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    __syncthreads();
  }

  // ---- the items: of whole lists a thread each, else a group of threads
  ChunkItem* items = reinterpret_cast<ChunkItem*>(a.ws + a.lay.items);
  ChunkMerge* merges = reinterpret_cast<ChunkMerge*>(a.ws + a.lay.merges);
  const int size = cut.whole == tiles || lists > 256 ? 1 : lists > 64 ? 4 : 32, sub = lane % size;  // threads a list
#pragma unroll 1
  for (int32_t u0 = 0; u0 < lists; u0 += kPlanThreads / size) {
    const int32_t u = u0 + tid / size;
    const bool on = u < lists;
    const int32_t t = on ? (int32_t)a.by_heads.div(u) : 0, h = on ? u - t * a.Hkv : 0;
    const Tile tl = t < kHeld ? tile[t] : load_tile(a, q, t);
    const Pieces p = pieces_of(cut, t, h, tl.g.n, t < kHeld ? before[t] : 0, a.Hkv);
    int32_t slot = -1;
    if (on && sub == 0) {
      atomicAdd(&n_items, p.count);
      if (p.count > 1) {
        slot = atomicAdd(&n_rows, p.count * tl.rows);
        atomicMax(&max_parts, p.count);
        merges[atomicAdd(&n_merges, 1)] = {h, tl.row0, tl.rows, tl.tok0, slot, p.count};
      }
    }
    slot = __shfl_sync(0xffffffffu, slot, lane - sub);
#pragma unroll 1
    for (int32_t i = sub; on && i < p.count; i += size) {
      const int32_t j0 = i == 0 ? 0 : p.first + (i - 1) * p.each;
      const int32_t j1 = i == 0 ? p.first : min(tl.g.n, j0 + p.each);
      const int32_t at = atomicAdd(equal ? &n_placed : &hist[bucket_of(j1 - j0)], 1);
      items[at] = {tl.request, h,          tl.row0, tl.rows,
                   j0,         j1,         tl.g.na, tl.g.shift,
                   slot < 0 ? -1 : slot + i * tl.rows, tl.tok0, tl.p0, tl.L};
    }
  }
  __syncthreads();
  if (tid == 0) {
    *chunk_head(a) = {n_items, n_merges, 0, most_rows, max_parts};
  }
  raise_flags(a.error_flags, eflags);
}

// out = sum of 2^(m_i - m) acc_i over the parts of a row, divided by the same sum of l_i.  A warp loads up to
// kAtOnce parts at once; a row with more is shared by up to 8 warps, each taking every so-manyth part.  Parts and
// warps are added in order, so the result is the same on every call.
constexpr int kAtOnce = 4;

template <typename T, int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkArgs a) {
  constexpr int E = D / 32;
  __shared__ float part_o[8][D], part_l[8], part_top[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // The attention kernel starts its CTAs' dependents once it has the plan, which is therefore readable already, from L2:
  // this kernel has not waited for it, so nothing says that older lines of it have left an SM's own cache.
  const int32_t* at = reinterpret_cast<const int32_t*>(chunk_head(a));
  const int32_t n_merges = __ldcg(at + 1), merge_rows = __ldcg(at + 3), merge_parts = __ldcg(at + 4);
  griddep_launch_dependents();
  if (n_merges == 0) {
    griddep_wait();
    return;
  }
  const int32_t n = n_merges * merge_rows;
  int share = merge_parts > 4 * kAtOnce   ? 8
              : merge_parts > 2 * kAtOnce ? 4
              : merge_parts > kAtOnce     ? 2
                                          : 1;  // warps a row: no more than there are
  while (share > 1 && n * (int64_t)share > 8 * gridDim.x) share /= 2;
  const int group = warp / share, which = warp % share, groups = 8 / share;
  const ChunkMerge* merges = reinterpret_cast<const ChunkMerge*>(a.ws + a.lay.merges);
  const float* ml = reinterpret_cast<const float*>(a.ws + a.lay.ml);
  const float* acc = reinterpret_cast<const float*>(a.ws + a.lay.acc);
  bool waited = false;
  for (int32_t u0 = blockIdx.x * groups; u0 < n; u0 += gridDim.x * groups) {
    const int32_t u = min(u0 + group, n - 1);
    const int4* note = reinterpret_cast<const int4*>(merges + u / merge_rows);
    const int4 tile = __ldcg(note);
    const int2 parts = __ldcg(reinterpret_cast<const int2*>(note + 1));
    const ChunkMerge m = {tile.x, tile.y, tile.z, tile.w, parts.x, parts.y};
    const int32_t row = u % merge_rows;
    const bool on = u0 + group < n && row < m.rows;
    if (!waited) griddep_wait();
    waited = true;
    float top = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int32_t p0 = which; on && p0 < m.parts; p0 += share * kAtOnce) {
      float2 x[kAtOnce];
      float f[kAtOnce][E];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int32_t p = p0 + i * share;
        x[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[i][e] = 0.f;
        if (p < m.parts) {
          const int64_t at = m.slot + (int64_t)p * m.rows + row;
          x[i] = *reinterpret_cast<const float2*>(ml + 2 * at);
          const float* v = acc + at * D + lane * E;
          if constexpr (E == 4) {
            const float4 y = *reinterpret_cast<const float4*>(v);
            f[i][0] = y.x, f[i][1] = y.y, f[i][2] = y.z, f[i][3] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2*>(v);
            f[i][0] = y.x, f[i][1] = y.y;
          }
        }
      }
      float now = top;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) now = fmaxf(now, x[i].x);
      const float ref = now == -INFINITY ? 0.f : now, w0 = fast_exp2(top - ref);
      l *= w0;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= w0;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const float w = fast_exp2(x[i].x - ref);
        l = fmaf(x[i].y, w, l);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(f[i][e], w, o[e]);
      }
      top = now;
    }
    if (share > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) part_o[warp][lane * E + e] = o[e];
      if (lane == 0) {
        part_l[warp] = l;
        part_top[warp] = top;
      }
      __syncthreads();
      if (which == 0) {
        float now = top;
        for (int w = 1; w < share; ++w) now = fmaxf(now, part_top[warp + w]);
        const float ref = now == -INFINITY ? 0.f : now;
        l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int w = 0; w < share; ++w) {
          const float x = fast_exp2(part_top[warp + w] - ref);
          l = fmaf(part_l[warp + w], x, l);
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = fmaf(part_o[warp + w][lane * E + e], x, o[e]);
        }
      }
      __syncthreads();
    }
    if (!on || which) continue;
    const int32_t rho = m.row0 + row;
    T* out = static_cast<T*>(a.out) +
             ((int64_t)(m.tok0 + rho / a.G) * a.Hq + m.head * a.G + rho % a.G) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = l == 0.f ? 0.f : o[e] / l;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < E; ++e) out[e] = o[e];
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = pack_bf16(o[e], o[e + 1]);
    }
  }
  if (!waited) griddep_wait();
}

}  // namespace

int32_t chunk_tile(const srkv_config& cfg) {
  return cfg.dtype == SRKV_BF16 ? kChunkTile : cfg.head_dim == 64 ? kChunkTileSimt64 : kChunkTileSimt128;
}

size_t chunk_workspace(const srkv_config& cfg, int32_t tokens, int32_t batch, ChunkLayout* out) {
  ChunkLayout w;
  const int64_t G = cfg.num_q_heads / cfg.num_kv_heads, Hkv = cfg.num_kv_heads;
  const int64_t tile = chunk_tile(cfg);
  const int64_t rows = (int64_t)tokens * cfg.num_q_heads;
  const int64_t some = batch < tokens ? batch : tokens;  // requests with a token
  const int64_t tiles = ((int64_t)tokens * G / tile + some) * Hkv;
  if (rows > INT32_MAX || tiles > INT32_MAX - 2 * kChunkSplitItems || batch > INT32_MAX / 2 - 1) return 0;
  w.items_cap = (int32_t)(tiles + ((kChunkSplitItems + Hkv - 1) / Hkv) * Hkv);
  w.merges_cap = kChunkSplitItems;
  const int64_t parts = rows * kChunkPartsPerRow;
  w.rows_cap = (int32_t)(parts < kChunkPartRows ? parts : kChunkPartRows);
  size_t off = align256(sizeof(ChunkHead));
  w.req = off;
  off = align256(off + sizeof(int32_t) * (2 * (size_t)batch + 2));
  w.items = off;
  off = align256(off + sizeof(ChunkItem) * (size_t)w.items_cap);
  w.merges = off;
  off = align256(off + sizeof(ChunkMerge) * (size_t)w.merges_cap);
  w.ml = off;
  off = align256(off + sizeof(float) * 2 * (size_t)w.rows_cap);
  w.acc = off;
  off = align256(off + sizeof(float) * (size_t)w.rows_cap * cfg.head_dim);
  w.total = off;
  if (out) *out = w;
  return w.total;
}

cudaError_t launch_chunk_plan(const ChunkArgs& a, cudaStream_t stream) {
  return launch_pdl(chunk_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
}

cudaError_t launch_chunk_merge(const ChunkArgs& a, int32_t dtype, cudaStream_t stream) {
  const dim3 g((unsigned)(4 * a.ctas)), b(256);
  if (dtype == SRKV_BF16)
    return a.d == 128 ? launch_pdl(chunk_merge_kernel<__nv_bfloat16, 128>, g, b, 0, stream, a)
                      : launch_pdl(chunk_merge_kernel<__nv_bfloat16, 64>, g, b, 0, stream, a);
  return a.d == 128 ? launch_pdl(chunk_merge_kernel<float, 128>, g, b, 0, stream, a)
                    : launch_pdl(chunk_merge_kernel<float, 64>, g, b, 0, stream, a);
}

}  // namespace srkv
