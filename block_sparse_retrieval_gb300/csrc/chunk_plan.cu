// chunk_plan.cu -- the plan of a chunk's attention, and the merge of divided tiles.
//
// Lengths live on the device, so the work is divided there: one CTA lists the items, longest first, and the
// attention kernel's CTAs take them one by one.  With many tiles no list is divided; with few, some ways of cutting
// the lists are tried, and the one with the least estimate is taken: the average load of a CTA, or, for the items of at
// least some size, the rounds that these need, whichever is most.
#include "chunk_plan.cuh"

namespace srkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kBuckets = 192;  // sizes 0 .. 7, then eight per octave
constexpr int kTrials = 8;
constexpr float kItemCost = 1.5f;  // what starting and ending an item costs, in pages
constexpr float kPartCost = 1.f;   // what a partial result adds

__device__ __forceinline__ int bucket_of(int32_t n) {
  if (n < 8) return n;
  const int e = 31 - __clz(n);
  return 8 * (e - 2) + ((n >> (e - 3)) & 7);
}
__device__ __forceinline__ int32_t size_of(int b) {  // the least size of a bucket
  return b < 8 ? b : (8 + (b & 7)) << (b / 8 - 1);
}

// How trial k divides the page lists: those of the first `whole` tiles not at all, the others, one behind the
// other (tile by tile, head by head), at every `grid` pages.  Trial 0 divides nothing.  Where lists are fewer than
// CTAs, the others divide all of them, into some fraction of an SM's load; else the first ones do, and the last ones
// divide what is left after full rounds of whole tiles.
struct Cuts {
  int32_t whole, grid;
};
__device__ __forceinline__ Cuts trial_cuts(int k, int32_t tiles, int32_t round_tiles, float avg, float rest_avg) {
  constexpr float few[kTrials] = {0.f, 1.5f, 1.2f, 1.f, .75f, .5f, .34f, .25f};
  constexpr float many[kTrials] = {0.f, 1.f, .5f, .25f, 1.f, .67f, .5f, .34f};
  if (k == 0) return {tiles, INT32_MAX};
  const bool rounds = round_tiles > 0 && k >= 4;
  const float n = ceilf((rounds ? rest_avg : avg) * (round_tiles > 0 ? many[k] : few[k]));
  return {rounds ? round_tiles : 0, n < 2.f ? 2 : n > 1e9f ? 1000000000 : (int32_t)n};
}

// The pieces of a list of n pages that starts at page `from` of the row of lists: the first one's end, and how
// many there are.
struct Pieces {
  int32_t first, count;
};
__device__ __forceinline__ Pieces pieces_of(long long from, int32_t n, int32_t grid) {
  const uint32_t into = from >> 32 ? (uint32_t)(from % grid) : (uint32_t)from % (uint32_t)grid;
  const int32_t to_cut = grid - (int32_t)into;
  if (n <= to_cut) return {n, 1};
  return {to_cut, 1 + (n - to_cut + grid - 1) / grid};
}

// The requests as the plan sees them: on chip while they are few, else in the workspace and the call's arrays.
struct Requests {
  const int32_t* first;  // first tile of each
  const int32_t* n;      // its new tokens (0: none, or refused)
  const int32_t* offset;
  const int32_t* len;
  int32_t count;
};
constexpr int kHeld = 512;  // requests, and tiles, that are held on chip

struct Tile {
  int32_t request, row0, rows, tok0, p0, L;
  ChunkPages g;
};

__device__ __forceinline__ Tile load_tile(const ChunkArgs& a, const Requests& q, int32_t tau) {
  Tile t;
  int32_t lo = 0, hi = q.count;  // the last request whose first tile is at or before tau
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (q.first[mid] <= tau)
      lo = mid;
    else
      hi = mid;
  }
  t.request = lo;
  const int32_t n = q.n[lo];
  t.row0 = (tau - q.first[lo]) * a.tile;
  t.rows = min(a.tile, n * a.G - t.row0);
  t.tok0 = q.offset[lo];
  t.L = (int32_t)min((int64_t)max(q.len[lo], 0), (int64_t)a.max_blocks * kBlock);
  t.p0 = t.L - n;
  t.g = chunk_pages(t.p0 + t.row0 / a.G, t.p0 + (t.row0 + t.rows - 1) / a.G, a.init, a.local);
  return t;
}

__device__ __forceinline__ ChunkItem make_item(const Tile& t, int32_t h, int32_t j0, int32_t j1, int32_t slot) {
  ChunkItem it;
  it.request = t.request;
  it.head = h;
  it.row0 = t.row0;
  it.rows = t.rows;
  it.j0 = j0;
  it.j1 = j1;
  it.na = t.g.na;
  it.shift = t.g.shift;
  it.slot = slot;
  it.tok0 = t.tok0;
  it.p0 = t.p0;
  it.L = t.L;
  return it;
}

template <typename I>
__device__ __forceinline__ I warp_scan(I v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkArgs a) {
  __shared__ int32_t hist[kTrials][kBuckets];
  __shared__ int32_t cursor[kBuckets];
  __shared__ int32_t held[4][kHeld];
  __shared__ Tile tile[kHeld];
  __shared__ long long before[kHeld];  // pages of the tiles before, for one head
  __shared__ unsigned long long part_rows[kTrials];
  __shared__ long long warp_sum[kPlanWarps];
  __shared__ int32_t split_items[kTrials], n_merges, n_rows, max_rows, max_parts;
  __shared__ float estimate[kTrials];
  __shared__ int32_t chosen;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kTrials * kBuckets; i += kPlanThreads) (&hist[0][0])[i] = 0;
  if (tid < kTrials) {
    part_rows[tid] = 0;
    split_items[tid] = 0;
  }
  if (tid == 0) {
    n_merges = 0;
    n_rows = 0;
    max_rows = 0;
    max_parts = 0;
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the requests' tiles
  const bool few = a.batch <= kHeld;
  int32_t* req = reinterpret_cast<int32_t*>(a.ws + a.lay.req);
  uint32_t eflags = 0;
  int32_t base = 0;
  const int32_t cap = a.lay.items_cap / a.Hkv - (kChunkSplitItems + a.Hkv - 1) / a.Hkv;  // tiles that good offsets make at most
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
    const long long tiles = ((int64_t)n * a.G + a.tile - 1) / a.tile;
    const long long x = warp_scan(tiles, lane);
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    long long first_tile = base, all = base;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
      const long long y = warp_sum[w];
      if (w < warp) first_tile += y;
      all += y;
    }
    if (r < a.batch) {
      // offsets that go back and forth could ask for more tiles than the workspace holds
      if (first_tile + x > cap) eflags |= SRKV_EFLAG_CHUNK;
      const int32_t first = (int32_t)min(first_tile + x - tiles, (long long)cap);
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
    base = (int32_t)min(all, (long long)cap);
    __syncthreads();
  }
  const int32_t tiles = base;
  const Requests q = {few ? held[0] : req, few ? held[1] : req + a.batch + 1, few ? held[2] : a.offsets,
                      few ? held[3] : a.seq_lens, a.batch};

  // ---- the load: pages of the lists, and of those before each tile
  long long sum = 0;
  for (int32_t t0 = 0; t0 < tiles; t0 += kPlanThreads) {
    const int32_t t = t0 + tid;
    int32_t n = 0;
    if (t < tiles) {
      const Tile tl = load_tile(a, q, t);
      n = tl.g.n;
      if (t < kHeld) tile[t] = tl;
    }
    const long long x = warp_scan((long long)n, lane);
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    long long at = sum;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
      if (w < warp) at += warp_sum[w];
      sum += warp_sum[w];
    }
    if (t < kHeld) before[t] = at + x - n;
    __syncthreads();
  }
  const float avg = (float)(sum * a.Hkv) / (float)a.ctas;
  // Lists are divided only where tiles are few: many balance by themselves.
  const int trials = tiles <= kHeld && tiles * (int64_t)a.Hkv < 16 * (int64_t)a.ctas ? kTrials : 1;
  const int32_t round_tiles = (int32_t)((int64_t)tiles * a.Hkv / a.ctas * a.ctas / a.Hkv);
  const float rest_avg = trials == 1 || round_tiles == tiles
                             ? 0.f
                             : (float)((sum - before[round_tiles]) * a.Hkv) / (float)a.ctas;

  // ---- the sizes that each trial gives: a thread per (list, trial)
  if (trials == 1) {
    for (int32_t t = tid; t < tiles; t += kPlanThreads)
      atomicAdd(&hist[0][bucket_of(t < kHeld ? tile[t].g.n : load_tile(a, q, t).g.n)], a.Hkv);
  } else {
    const int k = tid % kTrials;
    const Cuts cut = trial_cuts(k, tiles, round_tiles, avg, rest_avg);
    int32_t split = 0;
    unsigned long long all_rows = 0;
    for (int32_t u = tid / kTrials; u < tiles * a.Hkv; u += kPlanThreads / kTrials) {
      const int32_t t = u / a.Hkv, h = u - t * a.Hkv, n = tile[t].g.n;
      if (t < cut.whole) {
        atomicAdd(&hist[k][bucket_of(n)], 1);
        continue;
      }
      const Pieces p = pieces_of(before[t] * a.Hkv + (long long)h * n, n, cut.grid);
      atomicAdd(&hist[k][bucket_of(p.first)], 1);
      if (p.count > 1) {
        atomicAdd(&hist[k][bucket_of(n - p.first - (p.count - 2) * cut.grid)], 1);
        if (p.count > 2) atomicAdd(&hist[k][bucket_of(cut.grid)], p.count - 2);
        all_rows += (unsigned long long)p.count * tile[t].rows;
        split += p.count;
      }
    }
    if (split) {
      atomicAdd(&part_rows[k], all_rows);
      atomicAdd(&split_items[k], split);
    }
  }
  __syncthreads();

  // ---- each warp estimates one trial
  if (warp < trials) {
    float worst = 0.f, total = 0.f;
    int32_t seen = 0;
#pragma unroll
    for (int b0 = kBuckets - 32; b0 >= 0; b0 -= 32) {
      const int b = b0 + 31 - lane;  // the larger sizes first
      const int32_t n = hist[warp][b];
      if (!__any_sync(0xffffffffu, n != 0)) continue;
      const int32_t upto = seen + warp_scan(n, lane);
      const float cost = (float)size_of(b) + kItemCost;
      if (n > 0) worst = fmaxf(worst, (float)((upto + a.ctas - 1) / a.ctas) * cost);
      total += (float)n * cost;
      seen = __shfl_sync(0xffffffffu, upto, 31);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      worst = fmaxf(worst, __shfl_xor_sync(0xffffffffu, worst, o));
      total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane == 0) {
      const bool fits = part_rows[warp] <= (unsigned long long)a.lay.rows_cap &&
                        split_items[warp] <= kChunkSplitItems;
      const float est = fmaxf(worst, total / a.ctas) + (split_items[warp] > 0 ? kPartCost : 0.f);
      estimate[warp] = fits || warp == 0 ? est : 3e38f;
    }
  }
  __syncthreads();
  if (warp == 0) {
    float e = lane < trials ? estimate[lane] : INFINITY;
    int best = lane;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float f = __shfl_xor_sync(0xffffffffu, e, o);
      const int other = __shfl_xor_sync(0xffffffffu, best, o);
      if (f < e || (f == e && other < best)) {
        e = f;
        best = other;
      }
    }
    int32_t at = 0;
#pragma unroll
    for (int b0 = kBuckets - 32; b0 >= 0; b0 -= 32) {  // the longest items come first
      const int b = b0 + 31 - lane;
      const int32_t n = hist[best][b], upto = at + warp_scan(n, lane);
      cursor[b] = upto - n;
      at = __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) {
      chosen = best;
      ChunkHead* head = chunk_head(a);
      head->items = at;
      head->next = 0;
    }
  }
  __syncthreads();

  // ---- the items: of undivided lists a thread each, of divided ones a group of threads
  const Cuts cut = trial_cuts(chosen, tiles, round_tiles, avg, rest_avg);
  ChunkItem* items = reinterpret_cast<ChunkItem*>(a.ws + a.lay.items);
  ChunkMerge* merges = reinterpret_cast<ChunkMerge*>(a.ws + a.lay.merges);
  const int64_t whole = (int64_t)min(cut.whole, tiles) * a.Hkv;
  for (int64_t u = tid; u < whole; u += kPlanThreads) {
    const int32_t t = (int32_t)(u / a.Hkv), h = (int32_t)(u - (int64_t)t * a.Hkv);
    const Tile tl = t < kHeld ? tile[t] : load_tile(a, q, t);
    items[atomicAdd(&cursor[bucket_of(tl.g.n)], 1)] = make_item(tl, h, 0, tl.g.n, -1);
  }
  if (cut.whole < tiles) {
    const int32_t lists = (tiles - cut.whole) * a.Hkv;
    const int size = lists > 256 ? 4 : lists > 64 ? 8 : 32, sub = lane % size;  // threads a list
    for (int32_t u0 = 0; u0 < lists; u0 += kPlanThreads / size) {
      const int32_t u = u0 + tid / size;
      const bool on = u < lists;
      const int32_t t = cut.whole + (on ? u / a.Hkv : 0), h = on ? u % a.Hkv : 0;
      const Tile& tl = tile[t];
      const Pieces p = pieces_of(before[t] * a.Hkv + (long long)h * tl.g.n, tl.g.n, cut.grid);
      int32_t slot = -1;
      if (on && p.count > 1 && sub == 0) {
        slot = atomicAdd(&n_rows, p.count * tl.rows);
        atomicMax(&max_rows, tl.rows);
        atomicMax(&max_parts, p.count);
        ChunkMerge m;
        m.head = h;
        m.row0 = tl.row0;
        m.rows = tl.rows;
        m.tok0 = tl.tok0;
        m.slot = slot;
        m.parts = p.count;
        merges[atomicAdd(&n_merges, 1)] = m;
      }
      slot = __shfl_sync(0xffffffffu, slot, lane - sub);
      for (int32_t i = sub; on && i < p.count; i += size) {
        const int32_t j0 = i == 0 ? 0 : p.first + (i - 1) * cut.grid;
        const int32_t j1 = i == 0 ? p.first : min(tl.g.n, j0 + cut.grid);
        items[atomicAdd(&cursor[bucket_of(j1 - j0)], 1)] =
            make_item(tl, h, j0, j1, slot < 0 ? -1 : slot + i * tl.rows);
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    ChunkHead* head = chunk_head(a);
    head->merges = n_merges;
    head->merge_rows = max_rows;
    head->merge_parts = max_parts;
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
  // The attention kernel starts its CTAs' dependents once it has the plan, which is therefore readable already.
  const ChunkHead h = *chunk_head(a);
  griddep_launch_dependents();
  if (h.merges == 0) {
    griddep_wait();
    return;
  }
  const int share = h.merge_parts > 4 * kAtOnce   ? 8
                    : h.merge_parts > 2 * kAtOnce ? 4
                    : h.merge_parts > kAtOnce     ? 2
                                                  : 1;  // warps a row
  const int group = warp / share, which = warp % share, groups = 8 / share;
  const int32_t n = h.merges * h.merge_rows;
  const ChunkMerge* merges = reinterpret_cast<const ChunkMerge*>(a.ws + a.lay.merges);
  const float* ml = reinterpret_cast<const float*>(a.ws + a.lay.ml);
  const float* acc = reinterpret_cast<const float*>(a.ws + a.lay.acc);
  bool waited = false;
  for (int32_t u0 = blockIdx.x * groups; u0 < n; u0 += gridDim.x * groups) {
    const int32_t u = min(u0 + group, n - 1);
    const ChunkMerge m = merges[u / h.merge_rows];
    const int32_t row = u % h.merge_rows;
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
  return cfg.dtype == SRKV_BF16 ? kChunkTile : kChunkTileSimt;
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
