// rep_sums.cuh -- the one reduction behind every representation vector: the mean of a page's keys.
// Warp w sums its 16 rows [16w, 16w + 16) per 16-byte column chunk (a lane over the rows of its chunk, then
// warp shuffles across the lanes that hold the same chunk), and the 8 warp sums of a column are added in
// warp order.  The build at prefill and both appends share it, so that all give the same bits.
#pragma once

#include "srkv_internal.cuh"

namespace srkv {

constexpr int kRepWarps = 8;                 // warps that reduce a page
constexpr int kRepThreads = kRepWarps * 32;  // the append kernels' block
constexpr int kRepRingBytes = 192 * 1024;

template <typename T>
struct Vec16;  // 16 bytes of T, widened to float
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void widen(const int4& v, float (&f)[8]) {
    const uint32_t w[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  __device__ static void widen(const int4& v, float (&f)[4]) {
    f[0] = __int_as_float(v.x);
    f[1] = __int_as_float(v.y);
    f[2] = __int_as_float(v.z);
    f[3] = __int_as_float(v.w);
  }
};

// Geometry of one slab's reduction.
template <typename T, int D>
struct RepGeom {
  static constexpr int EPV = Vec16<T>::N;                  // elements per 16-byte chunk
  static constexpr int LPR = D / EPV;                      // chunks (lanes) per row
  static constexpr int RPI = 32 / LPR;                     // rows per warp-wide load
  static constexpr int RPW = kBlock / kRepWarps;           // rows per warp
  static constexpr int IPW = RPW / RPI;                    // loads per lane per slab
  static constexpr int CPW = D / kRepWarps;                // columns each warp finishes
  static constexpr int kSlab = kBlock * D * (int)sizeof(T);
  static constexpr int kStages = kRepRingBytes / kSlab;
  static_assert(LPR <= 32 && RPW % RPI == 0 && CPW <= 32, "slab geometry");
  // shared memory of the streaming kernel
  static constexpr size_t kOffPart = (size_t)kStages * kSlab;           // [stage][warp][D]
  static constexpr size_t kOffInfo = kOffPart + sizeof(float) * kStages * kRepWarps * D;
  static constexpr size_t kOffBar = kOffInfo + sizeof(int4) * kStages;  // full, ready, empty
  static constexpr size_t kSmem = kOffBar + sizeof(uint64_t) * 3 * kStages;
  static constexpr size_t kSmemAlloc = kSmem + 128;  // the ring starts 128-byte aligned
  static_assert(kSmemAlloc <= 232448, "shared memory opt-in limit");
};

// Adds a lane's 16 bytes of a row to its sums, one row after the other ...
template <typename T, int D>
__device__ __forceinline__ void add_row(const int4& raw, float (&acc)[RepGeom<T, D>::EPV]) {
  float f[RepGeom<T, D>::EPV];
  Vec16<T>::widen(raw, f);
#pragma unroll
  for (int e = 0; e < RepGeom<T, D>::EPV; ++e) acc[e] += f[e];
}
// ... and the lanes' sums of the same columns: lanes [0, LPR) get the sums of columns
// [lane * EPV, lane * EPV + EPV) (the other lanes hold copies).
template <typename T, int D>
__device__ __forceinline__ void across_rows(float (&acc)[RepGeom<T, D>::EPV]) {
  using R = RepGeom<T, D>;
#pragma unroll
  for (int o = R::LPR; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < R::EPV; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
}

// Warp `warp`'s sum over its rows r < v of the lane's column chunk: on return, lanes
// [0, LPR) hold the sums of columns [lane * EPV, lane * EPV + EPV) (the other lanes hold
// copies).  load(row, chunk) gives the 16 bytes of that chunk of that row.
template <typename T, int D, typename Load>
__device__ __forceinline__ void warp_column_sums(Load&& load, int warp, int lane, int32_t v,
                                                 float (&acc)[RepGeom<T, D>::EPV]) {
  using R = RepGeom<T, D>;
  const int chunk = lane % R::LPR, sub = lane / R::LPR;
  int4 raw[R::IPW];
#pragma unroll
  for (int i = 0; i < R::IPW; ++i) {
    const int row = warp * R::RPW + sub + i * R::RPI;
    raw[i] = row < v ? load(row, chunk) : make_int4(0, 0, 0, 0);
  }
#pragma unroll
  for (int e = 0; e < R::EPV; ++e) acc[e] = 0.f;
#pragma unroll
  for (int i = 0; i < R::IPW; ++i) add_row<T, D>(raw[i], acc);
  across_rows<T, D>(acc);
}

// part[w][c] = warp w's column sums; lanes [0, CPW) of warp `warp` finish columns
// [warp * CPW, warp * CPW + CPW): the 8 warp sums in warp order, divided by v.
template <typename T, int D>
__device__ __forceinline__ void finish_columns(const float* part, int warp, int lane, int32_t v,
                                               float* out) {
  using R = RepGeom<T, D>;
  if (lane < R::CPW) {
    const int c = warp * R::CPW + lane;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kRepWarps; ++w) s += part[w * D + c];
    out[c] = v > 0 ? s / (float)v : 0.f;
  }
}

template <typename T, int D>
__device__ __forceinline__ void store_column_sums(float* part, int warp, int lane,
                                                  const float (&acc)[RepGeom<T, D>::EPV]) {
  using R = RepGeom<T, D>;
  if (lane < R::LPR) {
#pragma unroll
    for (int e = 0; e < R::EPV; ++e) part[warp * D + lane * R::EPV + e] = acc[e];
  }
}

}  // namespace srkv
