// chunk_plan.cu -- the plan of a chunk's attention, and the merge of divided tiles.
//
// Lengths live on the device, so the work is divided there: one CTA lists the items, longest first, and the
// attention kernel's CTAs take them one by one.  With many tiles no list is divided; with few, lists are divided
// so that every SM has work: some lengths of an item are tried, and the one whose estimate (the longest of: the average load, and
// for every size the rounds that the items of at least that size need) is least is taken.
#include "chunk_plan.cuh"

namespace srkv {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kBuckets = 192;  // sizes 0 .. 7, then eight per octave
constexpr int kTrials = kPlanWarps;
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

// Length of an item under trial k, for an average load of `avg` pages a CTA; trial 0 divides nothing.
__device__ __forceinline__ int32_t trial_pages(int k, float avg) {
  constexpr float f[kTrials] = {0.f, 4.f,  2.f, 1.5f, 1.25f, 1.12f, 1.05f, 1.f,
                                .9f, .75f, .6f, .52f, .5f,   .36f,  .34f,  .25f};
  if (k == 0) return INT32_MAX;
  const float n = ceilf(avg * f[k]);
  return n < 1.f ? 1 : n > 1e9f ? 1000000000 : (int32_t)n;
}

// The requests as the plan sees them: on chip while they are few, else in the workspace and the call's arrays.
struct Requests {
  const int32_t* first;  // first tile of each
  const int32_t* n;      // its new tokens (0: none, or refused)
  const int32_t* offset;
  const int32_t* len;
  int32_t count;
};
constexpr int kHeld = kPlanThreads;  // requests, and tiles, that are held on chip

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
  __shared__ int32_t held[4][kHeld], pages[kHeld], rows[kHeld];
  __shared__ unsigned long long part_rows[kTrials], pages_sum;
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
    pages_sum = 0;
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
    long long before = base, all = base;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
      const long long y = warp_sum[w];
      if (w < warp) before += y;
      all += y;
    }
    if (r < a.batch) {
      // offsets that go back and forth could ask for more tiles than the workspace holds
      if (before + x > cap) eflags |= SRKV_EFLAG_CHUNK;
      const int32_t first = (int32_t)min(before + x - tiles, (long long)cap);
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

  // ---- the load
  unsigned long long sum = 0;
  for (int32_t t = tid; t < tiles; t += kPlanThreads) {
    const Tile tl = load_tile(a, q, t);
    sum += (unsigned long long)tl.g.n;
    if (t < kHeld) {
      pages[t] = tl.g.n;
      rows[t] = tl.rows;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0 && sum) atomicAdd(&pages_sum, sum * (unsigned long long)a.Hkv);
  __syncthreads();

  // ---- the sizes that each trial gives: a thread per (tile, trial)
  const float avg = (float)pages_sum / (float)a.ctas;
  const int trials = tiles * (int64_t)a.Hkv >= 8 * (int64_t)a.ctas ? 1 : kTrials;
  {
    const int k = trials == 1 ? 0 : tid % kTrials;
    const int32_t step = trials == 1 ? kPlanThreads : kPlanThreads / kTrials;
    const int32_t c = trial_pages(k, avg);
    int32_t split = 0;
    unsigned long long all_rows = 0;
    for (int32_t t = trials == 1 ? tid : tid / kTrials; t < tiles; t += step) {
      int32_t n, m;
      if (t < kHeld) {
        n = pages[t];
        m = rows[t];
      } else {
        const Tile tl = load_tile(a, q, t);
        n = tl.g.n;
        m = tl.rows;
      }
      const int32_t s = n > c ? (int32_t)(((uint32_t)n + c - 1) / (uint32_t)c) : 1;
      const int32_t each = s == 1 ? n : n / s, rest = n - each * s;  // `rest` items are one page longer
      atomicAdd(&hist[k][bucket_of(each)], (s - rest) * a.Hkv);
      if (rest) atomicAdd(&hist[k][bucket_of(each + 1)], rest * a.Hkv);
      if (s > 1) {
        all_rows += (unsigned long long)s * m * a.Hkv;
        split += s * a.Hkv;
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

  // ---- the items: a warp per tile, or every thread where tiles are few
  const int32_t c = trial_pages(chosen, avg);
  ChunkItem* items = reinterpret_cast<ChunkItem*>(a.ws + a.lay.items);
  ChunkMerge* merges = reinterpret_cast<ChunkMerge*>(a.ws + a.lay.merges);
  const bool wide = tiles < kPlanWarps / 2;
  __shared__ int32_t shared_slot[kPlanWarps][2];
  for (int32_t t = wide ? 0 : warp; t < tiles; t += wide ? 1 : kPlanWarps) {
    const Tile tl = load_tile(a, q, t);
    const int32_t s = tl.g.n > c ? (int32_t)(((uint32_t)tl.g.n + c - 1) / (uint32_t)c) : 1;
    const int32_t each = s == 1 ? tl.g.n : tl.g.n / s, rest = tl.g.n - each * s;
    int32_t slot = 0, merge = 0;
    if (s > 1) {
      if (wide ? tid == 0 : lane == 0) {
        shared_slot[t % kPlanWarps][0] = atomicAdd(&n_rows, s * tl.rows * a.Hkv);
        shared_slot[t % kPlanWarps][1] = atomicAdd(&n_merges, a.Hkv);
        atomicMax(&max_rows, tl.rows);
        atomicMax(&max_parts, s);
      }
      if (wide)
        __syncthreads();
      else
        __syncwarp();
      slot = shared_slot[t % kPlanWarps][0];
      merge = shared_slot[t % kPlanWarps][1];
      __syncwarp();
    }
    for (int32_t i = wide ? tid : lane; i < s * a.Hkv; i += wide ? kPlanThreads : 32) {
      const int32_t part = i / a.Hkv, h = i - part * a.Hkv;
      ChunkItem it;
      it.request = tl.request;
      it.head = h;
      it.row0 = tl.row0;
      it.rows = tl.rows;
      it.j0 = part * each + min(part, rest);
      it.j1 = it.j0 + each + (part < rest ? 1 : 0);
      it.na = tl.g.na;
      it.shift = tl.g.shift;
      it.slot = s > 1 ? slot + (h * s + part) * tl.rows : -1;
      it.tok0 = tl.tok0;
      it.p0 = tl.p0;
      it.L = tl.L;
      const int32_t at = atomicAdd(&cursor[bucket_of(it.j1 - it.j0)], 1);
      items[at] = it;
      if (part == 0 && s > 1) {
        ChunkMerge m;
        m.head = h;
        m.row0 = tl.row0;
        m.rows = tl.rows;
        m.tok0 = tl.tok0;
        m.slot = slot + h * s * tl.rows;
        m.parts = s;
        merges[merge + h] = m;
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

// out = sum of 2^(m_i - m) acc_i over the parts of a row, divided by the same sum of l_i.  A row with many parts is
// shared by up to 8 warps, each taking every so-manyth part, so that all loads are in flight at once; parts and
// warps are added in order, so the result is the same on every call.
template <typename T, int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkArgs a) {
  constexpr int E = D / 32;
  __shared__ float part_o[8][D], part_l[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // The attention kernel starts its CTAs' dependents once it has the plan, which is therefore readable already.
  const ChunkHead h = *chunk_head(a);
  griddep_launch_dependents();
  if (h.merges == 0) {
    griddep_wait();
    return;
  }
  const int share = h.merge_parts > 12 ? 8 : h.merge_parts > 6 ? 4 : h.merge_parts > 3 ? 2 : 1;  // warps a row
  const int group = warp / share, which = warp % share, groups = 8 / share;
  const int64_t n = (int64_t)h.merges * h.merge_rows;
  const ChunkMerge* merges = reinterpret_cast<const ChunkMerge*>(a.ws + a.lay.merges);
  const float* ml = reinterpret_cast<const float*>(a.ws + a.lay.ml);
  const float* acc = reinterpret_cast<const float*>(a.ws + a.lay.acc);
  bool waited = false;
  for (int64_t u0 = (int64_t)blockIdx.x * groups; u0 < n; u0 += (int64_t)gridDim.x * groups) {
    const int64_t u = u0 + group;
    const ChunkMerge m = merges[min(u, n - 1) / h.merge_rows];
    const int32_t row = (int32_t)(min(u, n - 1) % h.merge_rows);
    const bool on = u < n && row < m.rows;
    if (!waited) griddep_wait();
    waited = true;
    float top = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    if (on) {
      for (int32_t p = lane; p < m.parts; p += 32) {
        const float x = ml[2 * (int64_t)(m.slot + p * m.rows + row)];
        top = x > top ? x : top;
      }
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      if (top == -INFINITY) top = 0.f;
#pragma unroll 4
      for (int32_t p = which; p < m.parts; p += share) {
        const int64_t at = m.slot + p * m.rows + row;
        const float2 x = *reinterpret_cast<const float2*>(ml + 2 * at);
        const float w = fast_exp2(x.x - top);
        l = fmaf(x.y, w, l);
        const float* v = acc + at * D + lane * E;
        float f[E];
        if constexpr (E == 4) {
          const float4 y = *reinterpret_cast<const float4*>(v);
          f[0] = y.x, f[1] = y.y, f[2] = y.z, f[3] = y.w;
        } else {
          const float2 y = *reinterpret_cast<const float2*>(v);
          f[0] = y.x, f[1] = y.y;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(f[e], w, o[e]);
      }
    }
    if (share > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) part_o[warp][lane * E + e] = o[e];
      if (lane == 0) part_l[warp] = l;
      __syncthreads();
      if (which == 0) {
        for (int w = 1; w < share; ++w) {
          l += part_l[warp + w];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += part_o[warp + w][lane * E + e];
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
  const dim3 g((unsigned)(2 * a.ctas)), b(256);
  if (dtype == SRKV_BF16)
    return a.d == 128 ? launch_pdl(chunk_merge_kernel<__nv_bfloat16, 128>, g, b, 0, stream, a)
                      : launch_pdl(chunk_merge_kernel<__nv_bfloat16, 64>, g, b, 0, stream, a);
  return a.d == 128 ? launch_pdl(chunk_merge_kernel<float, 128>, g, b, 0, stream, a)
                    : launch_pdl(chunk_merge_kernel<float, 64>, g, b, 0, stream, a);
}

}  // namespace srkv
