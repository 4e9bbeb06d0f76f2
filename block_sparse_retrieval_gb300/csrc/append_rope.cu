// append_rope.cu -- a ragged chunk of new tokens into the paged cache, rotated to its positions on the way.
//
// Row i of request r's chunk stands at position p = seq_lens[r] + i.  Queries and keys are rotated by the
// angles p * freq_j (pairs of elements as planes), keys and values go to their pages, and the
// representation vector of every page written becomes the mean of its keys as held, in the order of
// rep_sums.cuh: the value a fresh build gives.
//
// Angles.  A frequency is held as the fraction of a turn per token in 64-bit fixed point, so p times it modulo
// 2^64 is the angle modulo one turn without any rounding: no position is too far.  The top 32 bits, less the
// nearest quarter turn, go through the Taylor series of sine and cosine on +-pi/4 in fp32 (terms up to x^9 and x^10:
// the next ones are below 2^-28 and 2^-31).  A 64-bit floating product would do the same at 1/64 of the fp32
// rate: some 30 us for 8192 tokens of 8 heads.
//
// Work.  One CTA per (page touched, kv head): its 8 warps go through the page's 128 rows, 16 each, the rows
// already there as read and the new ones as rotated, and sum them on the way, so that the vector needs no
// second read.  Other CTAs rotate the queries, a warp per token (or eight warps per token where tokens are
// few), with the token's angles computed once for all its heads.
//
// What bounds it.  8192 tokens of 32 / 8 heads: bytes; 201.6 MB in 35.3 us = 5.7 TB/s, 0.84 of the measured copy rate; in
// fp32 402.9 MB in 62.9 us, 0.94.
// 64 tokens: 5.2 us, three dependent reads (lengths, table, rows) and the launch; one token: 3.2 us.
#include "rep_sums.cuh"

namespace srkv {
namespace {

struct RopeArgs {
  const void* q;
  const void* k_new;
  const void* v_new;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const double* freqs;
  int32_t rope_dim, interleaved;
  void* q_out;
  void* k_cache;
  void* v_cache;
  int64_t num_pages;
  const int32_t* block_table;
  int32_t max_blocks;
  const int32_t* offsets;
  int32_t tokens;
  const int32_t* seq_lens;
  int32_t batch;
  float* reps;
  int32_t* error_flags;
  int32_t Hq, Hkv;
  int32_t kv_items;  // page items per kv head
  int32_t by_token;  // 1: item i is the page that token i opens for its request (few tokens a request)
  int32_t segs;      // warps per token of the query part
};

// First item of request r where items are counted by pages: a chunk of n tokens touches at most n / 128 + 2.
__device__ __forceinline__ int32_t page_base(int32_t offset, int32_t r) {
  return offset / kBlock + 2 * r;
}

// The last request whose first item is at or before x: 32 requests a round.  With one token a request, token x is
// request x's: looked at first, as each round waits for the one before.
__device__ __forceinline__ int32_t find_request(const RopeArgs& a, int32_t x, bool pages, int lane) {
  int32_t lo = 0, n = a.batch;
  if (!pages && x < n && a.offsets[x] == x && a.offsets[x + 1] == x + 1) return x;
  while (n > 1) {
    const int32_t step = (n + 31) / 32, i = lane * step;
    bool at = false;
    if (i < n) {
      const int32_t off = a.offsets[lo + i];
      at = (pages ? page_base(off, lo + i) : off) <= x;
    }
    const int32_t hit = 31 - __clz(__ballot_sync(0xffffffffu, at) | 1u);
    lo += hit * step;
    n = min(step, n - hit * step);
  }
  return lo;
}

struct Request {
  int32_t begin, n, past;  // rows [begin, begin + n) of the packed inputs, at positions past ...
  bool ok;
};

__device__ __forceinline__ Request load_request(const RopeArgs& a, int32_t r, uint32_t& eflags) {
  Request q;
  q.begin = a.offsets[r];
  const int32_t end = a.offsets[r + 1];
  q.past = a.seq_lens[r];
  q.n = end - q.begin;
  q.ok = true;
  if (q.begin < 0 || end < q.begin || end > a.tokens) {
    eflags |= SRKV_EFLAG_CHUNK;
    q.ok = false;
  } else if (q.n > 0 &&
             (q.past < 0 || (int64_t)q.past + q.n > (int64_t)a.max_blocks * kBlock)) {
    eflags |= SRKV_EFLAG_SEQ_LEN;
    q.ok = false;
  }
  return q;
}

// freq / (2 pi) modulo 1 in 64-bit fixed point; the product in twice 53 bits, as a fraction of many turns loses
// its leading bits.  A negative frequency is its opposite's complement: a small negative number's fraction would be
// next to 1, where 53 bits hold less of it.
__device__ __forceinline__ uint64_t turns_of(double freq) {
  constexpr double c = 0.15915494309189535, c_lo = -9.839338337591243e-18;  // 1 / (2 pi)
  const double f = fabs(freq), hi = f * c, lo = fma(f, c_lo, fma(f, c, -hi));
  const uint64_t turns = __double2ull_rn((hi - floor(hi)) * 18446744073709551616.0) +
                         (uint64_t)__double2ll_rn(lo * 18446744073709551616.0);
  return freq < 0. ? 0 - turns : turns;
}

// Sine and cosine of position p times a frequency (fraction of a turn, 64-bit fixed point).
__device__ __forceinline__ void sin_cos(int32_t p, uint64_t turns, float& s, float& c) {
  const uint64_t a = (uint64_t)(uint32_t)p * turns;
  const uint32_t top = (uint32_t)((a + 0x80000000ull) >> 32);
  const uint32_t quarter = (top + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(top - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float sn = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  sn = fmaf(z, sn, 8.3333333e-3f);
  sn = fmaf(z, sn, -1.6666667e-1f);
  sn = fmaf(x * z, sn, x);
  float cs = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  cs = fmaf(z, cs, -1.3888889e-3f);
  cs = fmaf(z, cs, 4.1666667e-2f);
  cs = fmaf(z, cs, -0.5f);
  cs = fmaf(z, cs, 1.f);
  const float ss = (quarter & 1) ? cs : sn, cc = (quarter & 1) ? sn : cs;
  s = (quarter & 2) ? -ss : ss;
  c = ((quarter + 1) & 2) ? -cc : cc;
}

__device__ __forceinline__ int4 pack(const float (&f)[8]) {
  return make_int4((int)pack_bf16(f[0], f[1]), (int)pack_bf16(f[2], f[3]),
                   (int)pack_bf16(f[4], f[5]), (int)pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ int4 pack(const float (&f)[4]) {
  return make_int4(__float_as_int(f[0]), __float_as_int(f[1]), __float_as_int(f[2]),
                   __float_as_int(f[3]));
}

// The part of a rotation that is the same for every row of a lane: which pairs its 16-byte chunk holds.
template <typename T, int D>
struct Rotor {
  using R = RepGeom<T, D>;
  static constexpr int E = R::EPV, N = E / 2;
  uint64_t turns[N];  // of the N angles that this lane computes for a row
  int partner;        // lane that holds the chunk's other elements (half split)
  bool on, low, inter;
  float cs[E], sn[E];  // of the row at hand, for each element; sn with its sign

  // `table`: turns of the rope_dim / 2 frequencies.
  __device__ __forceinline__ void init(const uint64_t* table, int rope_dim, bool interleaved, int lane) {
    const int chunk = lane % R::LPR, half = rope_dim / 2 / E;
    inter = interleaved;
    on = chunk < 2 * half;
    low = chunk < half;
    partner = !on ? lane : low ? lane + half : lane - half;
    const int j0 = interleaved ? chunk * N : (low ? chunk * E : (chunk - half) * E + N);
#pragma unroll
    for (int k = 0; k < N; ++k) turns[k] = on ? table[j0 + k] : 0;
  }

  // Every lane of the warp calls these two together.
  __device__ __forceinline__ void angles(int32_t p) {
    float s[N], c[N];
#pragma unroll
    for (int k = 0; k < N; ++k) sin_cos(p, turns[k], s[k], c[k]);
    if (inter) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        cs[2 * k] = cs[2 * k + 1] = c[k];
        sn[2 * k] = -s[k];
        sn[2 * k + 1] = s[k];
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {  // the lanes of a pair of chunks compute half of the angles each
      const float so = __shfl_sync(0xffffffffu, s[k], partner);
      const float co = __shfl_sync(0xffffffffu, c[k], partner);
      cs[k] = low ? c[k] : co;
      cs[N + k] = low ? co : c[k];
      sn[k] = low ? -s[k] : so;
      sn[N + k] = low ? -so : s[k];
    }
  }

  __device__ __forceinline__ int4 turn(const int4& x) const {
    float f[E], o[E], y[E];
    Vec16<T>::widen(x, f);
    if (inter) {
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = f[e ^ 1];
    } else {
      int4 w;
      w.x = __shfl_sync(0xffffffffu, x.x, partner);
      w.y = __shfl_sync(0xffffffffu, x.y, partner);
      w.z = __shfl_sync(0xffffffffu, x.z, partner);
      w.w = __shfl_sync(0xffffffffu, x.w, partner);
      Vec16<T>::widen(w, o);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = fmaf(o[e], sn[e], f[e] * cs[e]);
    return on ? pack(y) : x;
  }
};

// kDeep: all the old rows of a page are in flight at once (few tokens a request, where every wait shows);
// else two rows, in registers for four CTAs an SM (8192 tokens: 45.7 us with all rows, 38.5 with four, 35.4).
template <typename T, int D, bool kDeep>
__global__ void __launch_bounds__(kRepThreads, 4) append_rope_kernel(const RopeArgs a) {
  using R = RepGeom<T, D>;
  __shared__ float part[kRepWarps * D];
  __shared__ uint64_t table[D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = lane % R::LPR, sub = lane / R::LPR;
  uint32_t eflags = 0;
  griddep_wait();  // programmatic launch: the inputs may be the previous kernel's outputs
  griddep_launch_dependents();
  if (threadIdx.x < a.rope_dim / 2) table[threadIdx.x] = turns_of(a.freqs[threadIdx.x]);
  if (blockIdx.x == 0) {  // offsets that the search below may never meet
    for (int32_t r = threadIdx.x; r < a.batch; r += kRepThreads) load_request(a, r, eflags);
    raise_flags(a.error_flags, eflags);
    eflags = 0;
  }
  const int64_t kv_blocks = (int64_t)a.kv_items * a.Hkv;

  if (blockIdx.x >= kv_blocks) {
    // ------------------------------------------------------------------ queries
    __syncthreads();
    const int64_t unit = ((int64_t)blockIdx.x - kv_blocks) * kRepWarps + warp;
    const int32_t t = (int32_t)(unit / a.segs), seg = (int32_t)(unit % a.segs);
    if (t >= a.tokens) return;
    const int32_t r = find_request(a, t, false, lane);
    const Request rq = load_request(a, r, eflags);
    if (!rq.ok || t < rq.begin || t >= rq.begin + rq.n) return;
    Rotor<T, D> rot;
    rot.init(table, a.rope_dim, a.interleaved != 0, lane);
    rot.angles(rq.past + (t - rq.begin));
    const int32_t per = (a.Hq + a.segs - 1) / a.segs, h1 = min(a.Hq, (seg + 1) * per);
    const T* in = static_cast<const T*>(a.q) + (int64_t)t * a.q_stride;
    T* out = static_cast<T*>(a.q_out) + (int64_t)t * a.Hq * D;
    constexpr int kU = 4;  // loads in flight
    for (int32_t h0 = seg * per; h0 < h1; h0 += kU * R::RPI) {
      int4 x[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int32_t h = h0 + u * R::RPI + sub;
        x[u] = h < h1 ? reinterpret_cast<const int4*>(in + (int64_t)h * D)[chunk]
                      : make_int4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int32_t h = h0 + u * R::RPI + sub;
        const int4 y = rot.turn(x[u]);
        if (h < h1) reinterpret_cast<int4*>(out + (int64_t)h * D)[chunk] = y;
      }
    }
    return;
  }

  // ------------------------------------------------------------------ keys, values, the page's vector
  const int32_t item = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  const int32_t r = find_request(a, item, !a.by_token, lane);
  const Request rq = load_request(a, r, eflags);
  if (!rq.ok) return;
  int32_t block;
  if (a.by_token) {
    const int32_t i = item - rq.begin;
    if (i < 0 || i >= rq.n || (i > 0 && (rq.past + i) % kBlock != 0)) return;
    block = (rq.past + i) / kBlock;
  } else {
    const int32_t i = item - page_base(rq.begin, r);
    if (i < 0 || rq.n == 0) return;
    block = rq.past / kBlock + i;
    if ((int64_t)block * kBlock >= (int64_t)rq.past + rq.n) return;
  }
  const int32_t page = a.block_table[(int64_t)r * a.max_blocks + block];
  if (page < 0 || (int64_t)page >= a.num_pages) {
    if (threadIdx.x == 0) raise_flags(a.error_flags, SRKV_EFLAG_PAGE_RANGE);
    return;
  }
  __syncthreads();  // the table
  const int32_t first = rq.past - block * kBlock;  // the chunk's first row, in rows of this page
  const int32_t lo = max(first, 0), hi = min((int64_t)first + rq.n, (int64_t)kBlock);
  const int64_t slab = ((int64_t)page * a.Hkv + h) * (int64_t)kBlock * D;
  T* kc = static_cast<T*>(a.k_cache) + slab;
  T* vc = static_cast<T*>(a.v_cache) + slab;
  const T* kn = static_cast<const T*>(a.k_new) + (int64_t)h * D;
  const T* vn = static_cast<const T*>(a.v_new) + (int64_t)h * D;
  Rotor<T, D> rot;
  rot.init(table, a.rope_dim, a.interleaved != 0, lane);
  const int row0 = warp * R::RPW + sub;
  float acc[R::EPV];
#pragma unroll
  for (int e = 0; e < R::EPV; ++e) acc[e] = 0.f;
  // Row `row` rotated and written, with its value; what the cache holds of it.
  auto write = [&](int row, bool here, const int4& k, const int4& v) {
    rot.angles(block * kBlock + row);
    const int4 y = rot.turn(k);
    if (here) {
      reinterpret_cast<int4*>(kc + row * D)[chunk] = y;
      reinterpret_cast<int4*>(vc + row * D)[chunk] = v;
    }
    return y;
  };
  auto load_new = [&](int row, int4& k, int4& v) {
    const int64_t token = rq.begin + row - first;
    k = reinterpret_cast<const int4*>(kn + token * a.k_stride)[chunk];
    v = reinterpret_cast<const int4*>(vn + token * a.v_stride)[chunk];
  };
  if constexpr (kDeep) {
    // through shared memory, each lane its own pieces
    extern __shared__ int4 slab[];
    int4* own = slab + row0 * R::LPR + chunk;
#pragma unroll
    for (int i = 0; i < R::IPW; ++i) {
      const int row = row0 + i * R::RPI;
      if (row < lo)
        cp_async_16(smem_u32(own + i * R::RPI * R::LPR), reinterpret_cast<const int4*>(kc + row * D) + chunk);
      else if (row >= hi)
        own[i * R::RPI * R::LPR] = make_int4(0, 0, 0, 0);
    }
    const int warp0 = warp * R::RPW;
#pragma unroll 1
    for (int i = max(lo - warp0, 0) / R::RPI; i < R::IPW && warp0 + i * R::RPI < hi; ++i) {
      const int row = row0 + i * R::RPI;
      const bool here = row >= lo && row < hi;
      int4 k = make_int4(0, 0, 0, 0), v = k;
      if (here) load_new(row, k, v);
      const int4 y = write(row, here, k, v);
      if (here) own[i * R::RPI * R::LPR] = y;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int i = 0; i < R::IPW; ++i) add_row<T, D>(own[i * R::RPI * R::LPR], acc);
  } else {
    constexpr int kBatch = 2;
#pragma unroll 1
    for (int i0 = 0; i0 < R::IPW; i0 += kBatch) {
      if (row0 - sub + i0 * R::RPI >= hi) break;  // (for the whole warp)
      int4 raw[kBatch], v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int row = row0 + (i0 + i) * R::RPI;
        raw[i] = v[i] = make_int4(0, 0, 0, 0);
        if (row < lo)
          raw[i] = reinterpret_cast<const int4*>(kc + row * D)[chunk];
        else if (row < hi)
          load_new(row, raw[i], v[i]);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int row = row0 + (i0 + i) * R::RPI;
        const bool here = row >= lo && row < hi;
        if (__any_sync(0xffffffffu, here)) {
          const int4 y = write(row, here, raw[i], v[i]);
          if (here) raw[i] = y;
        }
        add_row<T, D>(raw[i], acc);
      }
    }
  }
  across_rows<T, D>(acc);
  store_column_sums<T, D>(part, warp, lane, acc);
  __syncthreads();
  finish_columns<T, D>(part, warp, lane, hi, a.reps + ((int64_t)page * a.Hkv + h) * D);
}

}  // namespace

cudaError_t launch_append_rope(const srkv_config& cfg, const void* q, int64_t q_stride,
                               const void* k_new, int64_t k_stride, const void* v_new,
                               int64_t v_stride, const int32_t* offsets, int32_t tokens,
                               const double* freqs, int32_t rope_dim, int32_t interleaved,
                               void* q_out, void* k_cache, void* v_cache, int64_t num_pages,
                               const int32_t* block_table, int32_t max_blocks,
                               const int32_t* seq_lens, int32_t batch, float* reps,
                               int32_t* error_flags, cudaStream_t stream) {
  RopeArgs a;
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.freqs = freqs;
  a.rope_dim = rope_dim;
  a.interleaved = interleaved;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_pages = num_pages;
  a.block_table = block_table;
  a.max_blocks = max_blocks;
  a.offsets = offsets;
  a.tokens = tokens;
  a.seq_lens = seq_lens;
  a.batch = batch;
  a.reps = reps;
  a.error_flags = error_flags;
  a.Hq = cfg.num_q_heads;
  a.Hkv = cfg.num_kv_heads;
  const int64_t by_pages = (int64_t)tokens / kBlock + 2 * (int64_t)batch;
  a.by_token = tokens <= by_pages;
  a.kv_items = (int32_t)(a.by_token ? tokens : by_pages);
  a.segs = tokens < 1024 ? kRepWarps : 1;
  const int64_t q_units = q ? (int64_t)tokens * a.segs : 0;
  const int64_t grid = (int64_t)a.kv_items * a.Hkv + (q_units + kRepWarps - 1) / kRepWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)grid), b(kRepThreads);
  const bool deep = a.by_token;
  const size_t slab = deep ? (size_t)kBlock * cfg.head_dim * (cfg.dtype == SRKV_BF16 ? 2 : 4) : 0;
  auto launch = [&](auto kernel) { return launch_pdl(kernel, g, b, slab, stream, a); };
  if (cfg.dtype == SRKV_BF16) {
    if (cfg.head_dim == 128)
      return deep ? launch(append_rope_kernel<__nv_bfloat16, 128, true>)
                  : launch(append_rope_kernel<__nv_bfloat16, 128, false>);
    return deep ? launch(append_rope_kernel<__nv_bfloat16, 64, true>)
                : launch(append_rope_kernel<__nv_bfloat16, 64, false>);
  }
  if (cfg.head_dim == 128) {
    // 64 KB of shared memory: the opt-in is set once per device (not during graph capture)
    static bool configured[128] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    if (deep && !configured[dev]) {
      e = cudaFuncSetAttribute(append_rope_kernel<float, 128, true>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)slab);
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
    return deep ? launch(append_rope_kernel<float, 128, true>) : launch(append_rope_kernel<float, 128, false>);
  }
  return deep ? launch(append_rope_kernel<float, 64, true>) : launch(append_rope_kernel<float, 64, false>);
}

}  // namespace srkv
