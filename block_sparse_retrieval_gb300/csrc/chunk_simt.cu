// chunk_simt.cu -- attention of a chunk over the paged cache on CUDA cores, in full precision: the fp32 path.
//
// A CTA takes a tile of 64 rows (128 at d 128) and walks its pages 64 tokens (32) at a time, the next ones on
// their way meanwhile: S = Q K^T by 8 rows x 4 tokens (2) of a thread, a running maximum and sum per row in fp32,
// O += P V by 8 rows x d / 16 columns of a thread, both in packed pairs of fp32.  Bound by the fp32 rate (4 d
// operations per row and token): 2048 tokens over 4096 more take 986 us, 41 TFLOP/s, its pipe busy on 58 % of the cycles;
// 8 warps an SM leave little to fall back on while a sum waits for its last term, so terms of one sum are kept apart
// (2 % faster).  7 ragged requests of up to 300 tokens at d 64 take 160 us, 31 TFLOP/s, the rest of which is the
// ends of chunks that fill a tile in part (195 with 4 rows x 4 tokens a thread, whose reads of shared memory took 24
// lines for 128 operations a lane instead of 16; 214 with tiles of 128 rows).  Rows are padded by 16 bytes so that
// a warp's tokens lie in different banks.
//
// Items of fewer rows (single tokens, the ends of chunks) would leave warps idle; there groups of warps share a step's
// 64 tokens, each with a maximum, a sum and outputs of its own, joined in order at the end; and a thread takes 4
// rows where 8 in all are enough.  64 single tokens over 4096 to 8192 each, 8 heads of 128: 2918 -> 880 us (3.7
// TB/s), of 64 835 -> 380 (4.2), bound by the reads of shared memory; 6 x 17 rows over up to 3712 tokens 167 -> 109.
#include "chunk_plan.cuh"

namespace srkv {
namespace {

template <int D>
struct SimtGeom {
  static constexpr int kRows = D == 64 ? kChunkTileSimt64 : kChunkTileSimt128;
  static constexpr int kThreads = 2 * kRows;
  static constexpr int LD = D + 4;  // padded row of Q, K and V
};

// The steps of an item: kPer rows of a thread, kRowWarps warps side by side over its rows; where there are more
// warps, groups of them share a step's tokens.
template <int D, int kPer, int kRowWarps>
struct Step {
  using S = SimtGeom<D>;
  static constexpr int kRows = 2 * kPer * kRowWarps;
  static constexpr int kWarps = S::kThreads / 32;
  static constexpr int kGroups = kWarps / kRowWarps < 4 ? kWarps / kRowWarps : 4;
  static constexpr bool kJoined = kGroups > 1;
  static constexpr int kTok = kJoined || D == 64 ? 64 : 32;  // tokens a step
  static constexpr int kWarpTok = kTok / kGroups;            // and a warp's, kCols of a thread
  static constexpr int kCols = kWarpTok / 16;
  static constexpr int LP = kTok + 4;
  static constexpr size_t kTile = sizeof(float) * kTok * S::LD;  // K and V: two of each, one in use and one on its way
  static constexpr size_t kQ = 0, kK = kQ + sizeof(float) * kRows * S::LD, kV = kK + 2 * kTile, kP = kV + 2 * kTile,
                          kSmem = kP + sizeof(float) * kRows * LP;
  // at a joined item's end, in place of K: each group's outputs, maxima and sums
  static constexpr size_t kAcc = kK, kMl = kAcc + sizeof(float) * kGroups * kRows * D;
  static_assert(!kJoined || kMl + sizeof(float) * 2 * kGroups * kRows <= kV, "the ends fit K's place");
};

constexpr float kHidden = -1.f;  // in place of a hidden token's weight

// acc += P V over n tokens; with kSkip some may be hidden, which are left out altogether (one may hold a NaN).
template <int D, int kPer, int kTokens, int LP, bool kSkip>
__device__ __forceinline__ void add_values(const float* sp, const float* sv, int ty, int tx,
                                           float2 (&acc)[kPer][D / 32]) {
  using S = SimtGeom<D>;
#pragma unroll 2
  for (int t = 0; t < kTokens; t += 4) {
    float4 v[4][D / 64];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        v[u][c] = *reinterpret_cast<const float4*>(sv + (t + u) * S::LD + c * 64 + tx * 4);
    float w[kPer][4];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float4 p = *reinterpret_cast<const float4*>(sp + (ty * kPer + i) * LP + t);
      w[i][0] = p.x, w[i][1] = p.y, w[i][2] = p.z, w[i][3] = p.w;
    }
    // a sum's terms as far apart as can be: products wait for those they depend on
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (kSkip && w[i][u] < 0.f) continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const float2 ww = make_float2(w[i][u], w[i][u]);
          acc[i][c * 2] = __ffma2_rn(ww, make_float2(v[u][c].x, v[u][c].y), acc[i][c * 2]);
          acc[i][c * 2 + 1] = __ffma2_rn(ww, make_float2(v[u][c].z, v[u][c].w), acc[i][c * 2 + 1]);
        }
      }
    }
  }
}

// Columns [col, col + 4) of a finished row: unnormalised to its partial result, or the output.
template <int D>
__device__ __forceinline__ void write_row(const ChunkArgs& a, const ChunkItem& it, int row, int col, const float4& x,
                                          float l) {
  if (it.slot >= 0) {
    float* acc = reinterpret_cast<float*>(a.ws + a.lay.acc) + (int64_t)(it.slot + row) * D + col;
    *reinterpret_cast<float4*>(acc) = x;
    return;
  }
  const int32_t rho = it.row0 + row, token = (int32_t)a.by_group.div(rho);
  float* out = static_cast<float*>(a.out) +
               ((int64_t)(it.tok0 + token) * a.Hq + it.head * a.G + (rho - token * a.G)) * D + col;
  const float w = 1.f / l;  // (without a finite logit zeros, whatever the values)
  *reinterpret_cast<float4*>(out) =
      l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * w, x.y * w, x.z * w, x.w * w);
}
__device__ __forceinline__ void write_statistics(const ChunkArgs& a, const ChunkItem& it, int row, float m, float l) {
  if (it.slot >= 0)
    *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.ws + a.lay.ml) + 2 * (int64_t)(it.slot + row)) =
        make_float2(m, l);
}

// One item; every thread of the CTA calls it.
template <int D, int kPer, int kRowWarps>
__device__ __forceinline__ void attend_item(const ChunkArgs& a, const ChunkItem& it, unsigned char* smem,
                                         uint32_t& eflags) {
  using S = SimtGeom<D>;
  using P = Step<D, kPer, kRowWarps>;
  constexpr int kThreads = S::kThreads, kTok = P::kTok, kCols = P::kCols;
  float* sq = reinterpret_cast<float*>(smem + P::kQ);
  const int tid = threadIdx.x, tx = tid % 16, group = tid / 32 / kRowWarps;
  const int ty = tid / 16 % (2 * kRowWarps);  // of the threads over the rows
  const int first = group * P::kWarpTok;      // the warp's first token of a step
  float* sp = reinterpret_cast<float*>(smem + P::kP) + first;
  const int32_t p_lo = it.p0 + (int32_t)a.by_group.div(it.row0),
                p_hi = it.p0 + (int32_t)a.by_group.div(it.row0 + it.rows - 1);
  for (int i = tid; i < P::kRows * (D / 4); i += kThreads) {
    const int row = i / (D / 4), c = i % (D / 4);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < it.rows) {
      const int32_t rho = it.row0 + row, token = (int32_t)a.by_group.div(rho);
      const float* q = static_cast<const float*>(a.q) + (int64_t)(it.tok0 + token) * a.q_stride +
                       (int64_t)(it.head * a.G + (rho - token * a.G)) * D;
      x = reinterpret_cast<const float4*>(q)[c];
    }
    *reinterpret_cast<float4*>(sq + row * S::LD + c * 4) = x;
  }
  const bool work = group < P::kGroups && (ty & ~1) * kPer < it.rows;  // the warp has tokens, and a row
  const int32_t rho0 = it.row0 + ty * kPer;
  float m[kPer], l[kPer];
  float2 acc[kPer][D / 32];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[i][e] = make_float2(0.f, 0.f);
  }
  // The next step to copy: tokens [t0, t0 + kTok) of position j of the list, whose page is `page`.
  auto page_at = [&](int32_t j) {
    return j < it.j1 ? a.block_table[(int64_t)it.request * a.max_blocks + (j < it.na ? j : j + it.shift)] : 0;
  };
  int32_t j = it.j0, t0 = 0, page = page_at(j), ahead = page_at(j + 1);
  auto turn_page = [&] {
    ++j;
    t0 = 0;
    page = ahead;
    ahead = page_at(j + 1);
  };
  auto seek = [&] {  // past pages that are not there
    while (j < it.j1 && (page < 0 || (int64_t)page >= a.num_pages)) {
      eflags |= SRKV_EFLAG_PAGE_RANGE;
      turn_page();
    }
    return j < it.j1;
  };
  auto copy = [&](int buffer) {
    const int32_t tok = (j < it.na ? j : j + it.shift) * kBlock + t0;
    const int64_t at = (((int64_t)page * a.Hkv + it.head) * kBlock + t0) * D;
    const float* k = static_cast<const float*>(a.k_cache) + at;
    const float* v = static_cast<const float*>(a.v_cache) + at;
    const uint32_t dk = smem_u32(smem + P::kK + buffer * P::kTile), dv = smem_u32(smem + P::kV + buffer * P::kTile);
#pragma unroll 4
    for (int i = tid; i < kTok * (D / 4); i += kThreads) {
      const int row = i / (D / 4), c = i % (D / 4);
      const uint32_t off = (row * S::LD + c * 4) * sizeof(float);
      const int n = tok + row < it.L ? 16 : 0;  // behind the sequence: zeros
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dk + off), "l"(k + row * D + c * 4), "r"(n)
                   : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dv + off), "l"(v + row * D + c * 4), "r"(n)
                   : "memory");
    }
  };
  bool more = seek();
  if (more) copy(0);
  for (int buffer = 0; more; buffer ^= 1) {
    const int32_t b = j < it.na ? j : j + it.shift, tok = b * kBlock + t0 + first;
    const bool masked = chunk_masked(b, p_lo, p_hi, a.init, a.local);
    const float* sk = reinterpret_cast<const float*>(smem + P::kK + buffer * P::kTile) + first * S::LD;
    const float* sv = reinterpret_cast<const float*>(smem + P::kV + buffer * P::kTile) + first * S::LD;
    t0 += kTok;
    if (t0 >= kBlock || b * kBlock + t0 > p_hi) turn_page();
    more = seek();
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // this step's tokens are there, and the last step's buffer is free
    if (more) copy(buffer ^ 1);
    if (work) {
      float2 s2[kPer][kCols];  // rows ty * 8 + i, tokens tx + 16 j: even and odd pairs of columns
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int jj = 0; jj < kCols; ++jj) s2[i][jj] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 k[kCols];
#pragma unroll
        for (int jj = 0; jj < kCols; ++jj)
          k[jj] = *reinterpret_cast<const float4*>(sk + (tx + 16 * jj) * S::LD + c);
        float4 q[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) q[i] = *reinterpret_cast<const float4*>(sq + (ty * kPer + i) * S::LD + c);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
          for (int jj = 0; jj < kCols; ++jj)
            s2[i][jj] = __ffma2_rn(make_float2(q[i].x, q[i].y), make_float2(k[jj].x, k[jj].y), s2[i][jj]);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
          for (int jj = 0; jj < kCols; ++jj)
            s2[i][jj] = __ffma2_rn(make_float2(q[i].z, q[i].w), make_float2(k[jj].z, k[jj].w), s2[i][jj]);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int32_t pos = it.p0 + (int32_t)a.by_group.div(rho0 + i);
        float top = m[i], s[kCols];
#pragma unroll
        for (int jj = 0; jj < kCols; ++jj) {
          s[jj] = (s2[i][jj].x + s2[i][jj].y) * a.scale_log2;
          if (masked && !chunk_attends(pos, tok + tx + 16 * jj, a.init, a.local)) s[jj] = -INFINITY;
          top = fmaxf(top, s[jj]);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ref = top == -INFINITY ? 0.f : top;
        const float w = exp2f(m[i] - ref);
        float sum = 0.f;
#pragma unroll
        for (int jj = 0; jj < kCols; ++jj) {
          const float p = exp2f(s[jj] - ref);
          sum += p;
          sp[(ty * kPer + i) * P::LP + tx + 16 * jj] = p;
        }
        m[i] = top;
        l[i] = fmaf(l[i], w, sum);  // of this thread's tokens: added up over the 16 threads at the end
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[i][e] = make_float2(acc[i][e].x * w, acc[i][e].y * w);
      }
      if (masked) {  // (apart from the weights: marked among them, pages that all rows see paid 3 % for it)
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
          const int32_t pos = it.p0 + (int32_t)a.by_group.div(rho0 + i);
#pragma unroll
          for (int jj = 0; jj < kCols; ++jj)
            if (!chunk_attends(pos, tok + tx + 16 * jj, a.init, a.local))
              sp[(ty * kPer + i) * P::LP + tx + 16 * jj] = kHidden;
        }
      }
      __syncwarp();  // a row's weights come from the 16 lanes that read them
      if (masked)
        add_values<D, kPer, P::kWarpTok, P::LP, true>(sp, sv, ty, tx, acc);
      else
        add_values<D, kPer, P::kWarpTok, P::LP, false>(sp, sv, ty, tx, acc);
    }
  }
  if (P::kJoined) __syncthreads();  // K is read
  if (work) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int row = ty * kPer + i;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4 x = make_float4(acc[i][c * 2].x, acc[i][c * 2].y, acc[i][c * 2 + 1].x, acc[i][c * 2 + 1].y);
        if (P::kJoined)
          *reinterpret_cast<float4*>(smem + P::kAcc + sizeof(float) * ((group * P::kRows + row) * D + c * 64 + tx * 4)) = x;
        else if (row < it.rows)
          write_row<D>(a, it, row, c * 64 + tx * 4, x, l[i]);
      }
      if (tx == 0) {
        if (P::kJoined)
          *reinterpret_cast<float2*>(smem + P::kMl + sizeof(float) * 2 * (group * P::kRows + row)) =
              make_float2(m[i], l[i]);
        else if (row < it.rows)
          write_statistics(a, it, row, m[i], l[i]);
      }
    }
  }
  if (!P::kJoined) return;
  // the groups' parts of each row, in their order
  __syncthreads();
  for (int i = tid; i < it.rows * (D / 4); i += kThreads) {
    const int row = i / (D / 4), col = i % (D / 4) * 4;
    const float2* ml = reinterpret_cast<const float2*>(smem + P::kMl) + row;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int g = 0; g < P::kGroups; ++g) top = fmaxf(top, ml[g * P::kRows].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < P::kGroups; ++g) {
      const float w = exp2f(ml[g * P::kRows].x - ref);
      const float4 y = *reinterpret_cast<const float4*>(smem + P::kAcc + sizeof(float) * ((g * P::kRows + row) * D + col));
      sum = fmaf(ml[g * P::kRows].y, w, sum);
      x = make_float4(fmaf(y.x, w, x.x), fmaf(y.y, w, x.y), fmaf(y.z, w, x.z), fmaf(y.w, w, x.w));
    }
    write_row<D>(a, it, row, col, x, sum);
    if (col == 0) write_statistics(a, it, row, top, sum);
  }
}

constexpr size_t larger(size_t x, size_t y) { return x > y ? x : y; }
template <int D>
constexpr size_t kSimtSmem = larger(larger(Step<D, 4, 1>::kSmem, Step<D, 8, 1>::kSmem),
                                    larger(larger(Step<D, 8, 2>::kSmem, Step<D, 8, 4>::kSmem),
                                           Step<D, 8, SimtGeom<D>::kThreads / 32>::kSmem));
static_assert(2 * (kSimtSmem<64> + 1024) <= 233472 && kSimtSmem<128> <= 232448, "two CTAs an SM; one");

template <int D>
__global__ void __launch_bounds__(SimtGeom<D>::kThreads, D == 64 ? 2 : 1) chunk_simt_kernel(const ChunkArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int32_t next;
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  ChunkHead* head = chunk_head(a);
  const int32_t n_items = head->items;
  const ChunkItem* items = reinterpret_cast<const ChunkItem*>(a.ws + a.lay.items);
  uint32_t eflags = 0;
  for (;;) {
    __syncthreads();
    if (tid == 0) next = atomicAdd(&head->next, 1);
    __syncthreads();
    if (next >= n_items) break;
    const ChunkItem it = items[next];
    if (it.rows <= 8)
      attend_item<D, 4, 1>(a, it, smem, eflags);
    else if (it.rows <= 16)
      attend_item<D, 8, 1>(a, it, smem, eflags);
    else if (it.rows <= 32)
      attend_item<D, 8, 2>(a, it, smem, eflags);
    else if (D == 64 || it.rows <= 64)
      attend_item<D, 8, 4>(a, it, smem, eflags);
    else
      attend_item<D, 8, SimtGeom<D>::kThreads / 32>(a, it, smem, eflags);
  }
  if (tid == 0) raise_flags(a.error_flags, eflags);
}

template <int D>
cudaError_t launch_d(const ChunkArgs& a, cudaStream_t stream) {
  // The shared-memory opt-in is set once per device (not during graph capture).
  static bool configured[128] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(chunk_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kSimtSmem<D>);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  return launch_pdl(chunk_simt_kernel<D>, dim3(a.ctas), dim3(SimtGeom<D>::kThreads), kSimtSmem<D>, stream, a);
}

}  // namespace

cudaError_t launch_chunk_simt(const ChunkArgs& a, cudaStream_t stream) {
  return a.d == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace srkv
