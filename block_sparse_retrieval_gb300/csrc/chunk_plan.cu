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

struct Tile {
  int32_t request, row0, rows, tok0, p0, L;
  ChunkPages g;
};

__device__ __forceinline__ Tile load_tile(const ChunkArgs& a, const int32_t* req, int32_t tau) {
  Tile t;
  int32_t lo = 0, hi = a.batch;  // the last request whose first tile is at or before tau
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (req[mid] <= tau)
      lo = mid;
    else
      hi = mid;
  }
  t.request = lo;
  const int32_t n = req[a.batch + 1 + lo];
  t.row0 = (tau - req[lo]) * a.tile;
  t.rows = min(a.tile, n * a.G - t.row0);
  t.tok0 = a.offsets[lo];
  const int32_t len = a.seq_lens[lo];
  t.L = (int32_t)min((int64_t)max(len, 0), (int64_t)a.max_blocks * kBlock);
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
  __shared__ unsigned long long part_rows[kTrials], pages_sum;
  __shared__ long long warp_sum[kPlanWarps];
  __shared__ int32_t split_items[kTrials], n_merges, n_rows, max_rows;
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
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the requests' tiles
  int32_t* req = reinterpret_cast<int32_t*>(a.ws + a.lay.req);
  uint32_t eflags = 0;
  int32_t base = 0;
  const int32_t cap = a.lay.items_cap / a.Hkv - (kChunkSplitItems + a.Hkv - 1) / a.Hkv;  // tiles that good offsets make at most
  __syncthreads();
  for (int32_t r0 = 0; r0 < a.batch; r0 += kPlanThreads) {
    const int32_t r = r0 + tid;
    int32_t n = 0;
    if (r < a.batch) {
      const int32_t s = a.offsets[r], e = a.offsets[r + 1], len = a.seq_lens[r];
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
    for (int w = 0; w < kPlanWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    if (r < a.batch) {
      // offsets that go back and forth could ask for more tiles than the workspace holds
      const bool fits = before + x <= cap;
      if (!fits) eflags |= SRKV_EFLAG_CHUNK;
      req[r] = (int32_t)min(before + x - tiles, (long long)cap);
      req[a.batch + 1 + r] = n;
    }
    base = (int32_t)min(all, (long long)cap);
    __syncthreads();
  }
  const int32_t tiles = base;
  __syncthreads();

  // ---- the load, and the sizes that each trial gives
  unsigned long long sum = 0;
  for (int32_t t = tid; t < tiles; t += kPlanThreads) sum += (unsigned long long)load_tile(a, req, t).g.n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) atomicAdd(&pages_sum, sum * (unsigned long long)a.Hkv);
  __syncthreads();
  const float avg = (float)((double)pages_sum / a.ctas);
  const int trials = tiles * (int64_t)a.Hkv >= 8 * (int64_t)a.ctas ? 1 : kTrials;
  for (int32_t t = tid; t < tiles; t += kPlanThreads) {
    const Tile tl = load_tile(a, req, t);
    for (int k = 0; k < trials; ++k) {
      const int32_t c = trial_pages(k, avg);
      const int32_t s = tl.g.n > c ? (tl.g.n + c - 1) / c : 1;
      const int32_t rest = tl.g.n % s;  // items one page longer
      atomicAdd(&hist[k][bucket_of(tl.g.n / s)], (s - rest) * a.Hkv);
      if (rest) atomicAdd(&hist[k][bucket_of(tl.g.n / s + 1)], rest * a.Hkv);
      if (s > 1) {
        atomicAdd(&part_rows[k], (unsigned long long)s * tl.rows * a.Hkv);
        atomicAdd(&split_items[k], s * a.Hkv);
      }
    }
  }
  __syncthreads();

  // ---- each warp estimates one trial
  if (warp < trials) {
    float worst = 0.f, total = 0.f;
    int32_t seen = 0;
    for (int b0 = kBuckets - 32; b0 >= 0; b0 -= 32) {
      const int b = b0 + 31 - lane;  // the larger sizes first
      const int32_t n = hist[warp][b];
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
      float est = fmaxf(worst, total / a.ctas) + (split_items[warp] > 0 ? kPartCost : 0.f);
      estimate[warp] = fits || warp == 0 ? est : 3e38f;
    }
  }
  __syncthreads();
  if (tid == 0) {
    int best = 0;
    for (int k = 1; k < trials; ++k)
      if (estimate[k] < estimate[best]) best = k;
    chosen = best;
    int32_t at = 0;
    for (int b = kBuckets - 1; b >= 0; --b) {  // the longest items come first
      cursor[b] = at;
      at += hist[best][b];
    }
    ChunkHead* head = chunk_head(a);
    head->items = at;
    head->next = 0;
  }
  __syncthreads();

  // ---- the items: a warp per tile
  const int32_t c = trial_pages(chosen, avg);
  ChunkItem* items = reinterpret_cast<ChunkItem*>(a.ws + a.lay.items);
  ChunkMerge* merges = reinterpret_cast<ChunkMerge*>(a.ws + a.lay.merges);
  for (int32_t t = warp; t < tiles; t += kPlanWarps) {
    const Tile tl = load_tile(a, req, t);
    const int32_t s = tl.g.n > c ? (tl.g.n + c - 1) / c : 1;
    const int32_t rest = tl.g.n % s, each = tl.g.n / s;
    int32_t slot = 0, merge = 0;
    if (s > 1 && lane == 0) {
      slot = atomicAdd(&n_rows, s * tl.rows * a.Hkv);
      merge = atomicAdd(&n_merges, a.Hkv);
      atomicMax(&max_rows, tl.rows);
    }
    slot = __shfl_sync(0xffffffffu, slot, 0);
    merge = __shfl_sync(0xffffffffu, merge, 0);
    for (int32_t i = lane; i < s * a.Hkv; i += 32) {
      const int32_t part = i / a.Hkv, h = i % a.Hkv;
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
  }
  raise_flags(a.error_flags, eflags);
}

// One warp per row of a divided tile: out = sum of 2^(m_i - m) acc_i over the parts, divided by the same sum of
// l_i.  Parts are taken in order, so the result is the same on every call.
template <typename T, int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), warps = (int64_t)gridDim.x * 8;
  const int32_t n = chunk_head(a)->merges, most = chunk_head(a)->merge_rows;
  const ChunkMerge* merges = reinterpret_cast<const ChunkMerge*>(a.ws + a.lay.merges);
  const float* ml = reinterpret_cast<const float*>(a.ws + a.lay.ml);
  const float* acc = reinterpret_cast<const float*>(a.ws + a.lay.acc);
  constexpr int E = D / 32;
  for (int64_t u = warp; u < (int64_t)n * most; u += warps) {
    const ChunkMerge m = merges[u / most];
    const int32_t row = (int32_t)(u % most);
    if (row >= m.rows) continue;
    float top = -INFINITY;
    for (int32_t p = lane; p < m.parts; p += 32) {
      const float x = ml[2 * (int64_t)(m.slot + p * m.rows + row)];
      top = x > top ? x : top;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == -INFINITY) top = 0.f;
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int32_t p = 0; p < m.parts; ++p) {
      const int64_t at = m.slot + p * m.rows + row;
      const float2 x = *reinterpret_cast<const float2*>(ml + 2 * at);
      const float w = fast_exp2(x.x - top);
      l = fmaf(x.y, w, l);
      const float* v = acc + at * D + lane * E;
      float f[E];
      if constexpr (E == 4) {
        const float4 q = *reinterpret_cast<const float4*>(v);
        f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
      } else {
        const float2 q = *reinterpret_cast<const float2*>(v);
        f[0] = q.x, f[1] = q.y;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f[e], w, o[e]);
    }
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
