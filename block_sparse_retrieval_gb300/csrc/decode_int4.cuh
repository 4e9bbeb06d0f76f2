// decode_int4.cuh -- the decode's stages over 4-bit pages (int4_page.cuh): the ring between the
// producer warp and the consumers, the consumers' attention, and the merger of their states.
//
// softmax(q K^T / sqrt(d)) V with K = klo_t + ks_t ck_td and V = vlo_t + vs_t cv_td (token t, element
// d, codes c in 0..15):
//   logit_t = ks_t (sum_d q_d ck_td) + klo_t (sum_d q_d),
//   out_d   = sum_t (w_t vs_t) cv_td + sum_t w_t vlo_t,     w_t = softmax weight,
// so both products take the bare codes and a row's scale and minimum enter once per (token, head).
//
// What bounds it: per token and kv head 136 bytes arrive (d 128; an SM's share of the bandwidth
// brings them in 5.8 cycles) and 256 codes have to become matrix operands, so a code may cost a few
// instructions of an SM's 4 a cycle and no more.  The products are m16n8k16 ones with the group's
// heads as the N = 8 side, fed from registers: tensor memory would need the codes widened in shared
// memory first.  A code costs 5/8 of an instruction here: a word masked with 0x000f000f or 0x00f000f0
// is two fp16 subnormals, code * 2^-24 or code * 2^-20, operands as they are (subnormals are exact
// there), and one shift per word reaches the other four.  The powers of two are taken out of the query
// (16 times smaller at the second kind's elements) and of the weights likewise.
// Measured: dense batch 4 x 131072 (570 MB of slabs) 100 us, 84 % of the copy peak, 13.0 instructions
// a token and kv head; an SM issues on 46 % of its cycles and its warps wait for pages a third of the
// time.  At top-k 0.2 41.5 us (57 %): the scoring and the
// launches around the 23 us of bytes.  The 65536-token layer 13.6 us in one kernel, of which 3.4 are bytes.
// Groups of 8 heads: dense 111 us (76 %, 14.2 instructions), 42.2 and 14.4.
//
// A page is 4 groups of 32 tokens, one for each warp of a group of 4; the CTA's groups work on
// consecutive stages (3 of them, 2 for groups of more than 4 heads), so that 3 warps share a scheduler
// and hide one another's latencies (8 warps of 64 tokens: 135 us against 105 in the dense case; 16 of
// 32 with 96 registers: 146).  A group visits its own stages only.  Stages name their segment (a
// unit's positions in a list) by its number; a warp that meets a new number leaves its state
// of the old segment in shared memory and goes on at once, and a merger warp joins the states and
// writes the partial.  (Draining the groups and merging in them cost 5 us a segment.)
// Lane (g, t) of a warp (g = lane / 4):
//   S^T = K . Q^T, two 16-token tiles j per 32 tokens: tile row m holds token 8 (m / 2) + 4 j + (m & 1)
//     for m < 8 and that + 2 for row m + 8, so that rows 2t, 2t + 1, 2t + 8, 2t + 9 are the four
//     tokens whose nibbles sit in bits 8j .. 8j + 7 of both halves of octet t's value words: the
//     weights of S^T feed O^T = V^T . P without moving between lanes but for one movmatrix each;
//   V^T: lane (g, t) reads the words of octet t for elements 4g + 32x .. + 3 (one 16-byte load), two
//     to a 16-row tile.
// Both layouts make every 8-lane phase of the 16-byte shared loads contiguous (128 bytes).
//
// Groups of at most 4 heads leave half of the 8 columns of S^T free.  Columns 4..7 then repeat
// the heads 0..3, so that lanes t and t + 2 hold the same heads and each takes one of the two rows
// (g, g + 8) through the softmax: half the work per lane.  One movmatrix turns both rows' weights at
// once (columns 4..7 come out as the rows g + 8 of heads 0..3), a shuffle brings the second half over.
//
// Online softmax with a lazy reference: the weights are 2^(s - m) for a reference m that is raised
// only when some s exceeds it by 2^8, which a vote finds.  Likewise the fp16 operand of the second
// product, weight * vs * 2^11 / lim, has a power of two lim for each head that is raised when some operand
// passes 2^15 (the same vote).  Then the accumulators are rescaled.  lim follows the products and not
// the scales: a row with a large scale and next to no weight would otherwise press the other rows'
// operands below fp16's range.  When the weights' reference rises, lim falls with them.
#pragma once

#include "decode_mma.cuh"
#include "int4_page.cuh"

namespace srkv {

constexpr float kInt4Headroom = 8.f;   // log2 of the most a weight may exceed its reference
// log2 of the fp16 operand at weight * vs = lim: room for products 16 times larger before lim is raised
// (14, room for 2: 65536-token layer 13.55 -> 13.8 us, dense 99.8 -> 100.7), and the largest product met is
// 2^10 at least, so that 11 bits stay down to 2^-24 of it (rows g + 8: 2^-20).
constexpr int kInt4PLog2 = 11;
constexpr int kMergerWarp = kProducerWarp + 1;  // warps past it are consumers 8, 9, ...

struct alignas(16) Int4Stage {  // two 16-byte loads
  int32_t seg;   // number of the segment
  int32_t last;  // 1: no page and no stage behind it; every segment below `seg` is over
  int32_t lo, hi, ie, ws;
  int32_t pad[2];
};
struct Int4Segment {
  int32_t unit, flags;  // kBankB
};

// A stage is one slab (17 408 bytes at d 128), moved by one bulk copy.
template <int D, bool kNarrow>
struct Int4Cfg {
  static constexpr int kHeads = kNarrow ? 4 : 8;  // of a group, at most
  static constexpr int kSlab = Int4Slab<D>::kBytes;
  static constexpr int kGroupWarps = 4;           // warps that share a stage
  static constexpr int kWarps = kNarrow ? 12 : 8;  // consumer warps
  static constexpr int kGroups = kWarps / kGroupWarps;
  static constexpr int kThreads = (kWarps + 2) * 32;  // + the producer and the merger
  static constexpr int kStages = D == 128 ? (kNarrow ? 9 : 8) : (kNarrow ? 18 : 16);
  // A group waits for its own stages only, so each slot of the ring has to be one group's: a wait by
  // parity takes the phase before the current one for complete, and would pass at once on a slot
  // whose last use, another group's, has not landed.
  static_assert(kStages % kGroups == 0, "a ring slot belongs to one group");
  // A warp may be one stage of its group plus the ring behind the producer.
  static constexpr int kSegs = kStages + kGroups;
  static constexpr int kQBytes = kHeads * D * 2;
  static constexpr int MT = D / 16;
  // A warp's state in shared memory: (m, l) and acc of the lanes that hold heads.
  static constexpr int kStateStride = MT * 4 + 4;
  static constexpr int kState = (kNarrow ? 16 : 32) * kStateStride;

  static constexpr size_t kOffK = 0;
  static constexpr size_t kOffQ = (size_t)kStages * kSlab;
  // the one-kernel decode's leader streams no pages and keeps its partials from here on
  static constexpr size_t kOffV = (size_t)(kStages / 2) * kSlab;
  static constexpr size_t kOffState = kOffQ + (size_t)kSegs * kQBytes;
  static constexpr size_t kOffInfo = kOffState + sizeof(float) * kWarps * kState;
  static constexpr size_t kOffSeg = kOffInfo + sizeof(Int4Stage) * kStages;
  static constexpr size_t kOffBar = kOffSeg + ((sizeof(Int4Segment) * kSegs + 15) & ~size_t(15));
  // full[kStages], empty[kStages], query[kSegs], left (a segment's states), merged; then `done`
  static constexpr int kBars = 2 * kStages + kSegs + 2;
  static constexpr size_t kOffDone = kOffBar + sizeof(uint64_t) * kBars;
  static constexpr size_t kSmem = kOffDone + 16;
  static constexpr size_t kSmemAlloc = kSmem + 1024;
  static_assert(kSmemAlloc <= 232448, "shared memory opt-in limit");
};
template <int D>
struct Cfg<D, kInt4Narrow> : Int4Cfg<D, true> {};
template <int D>
struct Cfg<D, kInt4Wide> : Int4Cfg<D, false> {};

// 2^n, and 1 / f of a power of two f (normal numbers both).
__device__ __forceinline__ constexpr float exp2_of(int n) {
  return n < 0 ? 1.f / (float)(1ull << -n / 2) / (float)(1ull << (-n + 1) / 2)
               : (float)(1ull << n / 2) * (float)(1ull << (n + 1) / 2);
}
__device__ __forceinline__ float inverse_exp2(float f) {
  return __uint_as_float(0x7f000000u - __float_as_uint(f));
}

// The larger of each half (NaN if one is).
__device__ __forceinline__ uint32_t max_f16x2(uint32_t x, uint32_t y) {
  const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2*>(&x),
                                *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&m);
}

template <int D, int Fmt>
struct Int4Ring {
  using C = Cfg<D, Fmt>;
  unsigned char* smem;
  __device__ __forceinline__ uint64_t* full(int s) const { return bars() + s; }
  __device__ __forceinline__ uint64_t* empty(int s) const { return bars() + C::kStages + s; }
  __device__ __forceinline__ uint64_t* query(int s) const { return bars() + 2 * C::kStages + s; }
  __device__ __forceinline__ uint64_t* left() const { return query(C::kSegs); }
  __device__ __forceinline__ uint64_t* merged() const { return query(C::kSegs) + 1; }
  __device__ __forceinline__ Int4Stage* stage(int s) const {
    return reinterpret_cast<Int4Stage*>(smem + C::kOffInfo) + s;
  }
  __device__ __forceinline__ Int4Segment* segment(int s) const {
    return reinterpret_cast<Int4Segment*>(smem + C::kOffSeg) + s;
  }
  __device__ __forceinline__ volatile int32_t* done() const {
    return reinterpret_cast<volatile int32_t*>(smem + C::kOffDone);
  }
  __device__ __forceinline__ unsigned char* slab(int s) const {
    return smem + C::kOffK + (size_t)s * C::kSlab;
  }
  __device__ __forceinline__ unsigned char* q(int s) const {
    return smem + C::kOffQ + (size_t)s * C::kQBytes;
  }
  __device__ __forceinline__ float* state(int floats) const {
    return reinterpret_cast<float*>(smem + C::kOffState) + floats;
  }
  // Barrier set-up (a whole warp: one thread's 32 would stand before every decode's first copy).
  __device__ __forceinline__ void init(int lane) const {
    for (int i = lane; i < C::kBars; i += 32) {
      const bool is_empty = i >= C::kStages && i < 2 * C::kStages;
      const bool is_left = bars() + i == left();
      mbar_init(bars() + i, is_empty  ? C::kGroupWarps
                            : is_left ? C::kWarps
                                      : 1);
    }
    if (lane == 0) *done() = 0;
    fence_mbar_init();
  }

 private:
  __device__ __forceinline__ uint64_t* bars() const {
    return reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  }
};

// The producer's place: stages and segments handed out so far (uniform over its warp).
struct Int4Place {
  int64_t it = 0;
  int32_t segs = 0;
  int32_t queries = 0;  // of them with a query copied
  bool abort = false;
};

// Hands the pages of lanes [first, last) to the consumers, in lane order (the whole producer warp
// calls it): the lane's page is task t of unit u; kNewUnit in fl opens a segment, kBankB says of which
// list.  Each lane issues its own page.  A 4-bit page lasts an SM 0.4 us, so what a page costs the
// producer counts: everything but the wait for the stage, its description and the copy is computed by
// the lanes side by side (one lane for all: 0.75 us a page, 161 us in the dense case).
template <int D, int Fmt>
__device__ __forceinline__ void issue_batch_int4(const DecodeArgs& a, unsigned char* smem,
                                                 Int4Place& pl, int first, int last, int32_t u,
                                                 uint32_t fl, const PageTask& t, uint32_t& eflags,
                                                 int lane) {
  using C = Cfg<D, Fmt>;
  const Int4Ring<D, Fmt> ring{smem};
  const int64_t mine = pl.it + (lane - first);
  const int s = (int)(mine % C::kStages);
  const uint32_t parity = (uint32_t)((mine / C::kStages - 1) & 1);
  const bool rows = t.page >= 0 && t.hi > t.lo;
  const bool fresh = lane >= first && lane < last && (fl & kNewUnit) != 0;
  const uint32_t opens = __ballot_sync(0xffffffffu, fresh);
  const int32_t seg = pl.segs + __popc(opens & (0xffffffffu >> (31 - lane))) - 1;
  const int32_t h = u % a.Hkv, r = u / a.Hkv;
  const uint32_t qbytes = (uint32_t)(a.G * D * 2);
  const unsigned char* src = static_cast<const unsigned char*>(a.k_cache) +
                             ((int64_t)(rows ? t.page : 0) * a.Hkv + h) * C::kSlab;
  const __nv_bfloat16* q =
      static_cast<const __nv_bfloat16*>(a.q) + ((int64_t)r * a.Hq + (int64_t)h * a.G) * D;
  const uint64_t once = l2_policy_evict_first();  // pages are read once per step
  for (int l = first; l < last && !pl.abort; ++l) {
    bool ok = true;
    if (lane == l) {
      ok = mine < C::kStages || mbar_wait(ring.empty(s), parity);
      if (ok) {
        if (fresh) {  // (the slot of segment seg - kSegs: every warp is past it, see kSegs)
          const int qslot = seg % C::kSegs;
          *ring.segment(qslot) = Int4Segment{u, (int32_t)(fl & kBankB)};
          mbar_arrive_expect_tx(ring.query(qslot), qbytes);
          bulk_load(ring.q(qslot), q, qbytes, ring.query(qslot));
        }
        int4* info = reinterpret_cast<int4*>(ring.stage(s));
        info[0] = make_int4(seg, 0, rows ? t.lo : 0, rows ? t.hi : 0);
        info[1] = make_int4(t.ie, t.ws, 0, 0);
        mbar_arrive_expect_tx(ring.full(s), rows ? (uint32_t)C::kSlab : 0u);
        if (rows) bulk_load_hint(ring.slab(s), src, (uint32_t)C::kSlab, ring.full(s), once);
      }
    }
    __syncwarp();  // a segment's entry is written before any later stage of it is handed out
    if (__all_sync(0xffffffffu, ok)) {
      ++pl.it;
    } else {  // the caller still waits (bounded) for the copies already started
      pl.abort = true;
      eflags |= SRKV_EFLAG_TIMEOUT;
    }
  }
  pl.segs += __popc(opens);
  pl.queries += __popc(opens);
}

// The end: a stage for each group that closes every segment, then every copy lands.
template <int D, int Fmt>
__device__ __forceinline__ void finish_ring_int4(unsigned char* smem, Int4Place& pl,
                                                 uint32_t& eflags, int lane) {
  using C = Cfg<D, Fmt>;
  const Int4Ring<D, Fmt> ring{smem};
  if (lane != 0) return;
  for (int g = 0; g < C::kGroups && !pl.abort; ++g) {
    const int s = (int)(pl.it % C::kStages);
    if (pl.it >= C::kStages && !mbar_wait(ring.empty(s), (uint32_t)((pl.it / C::kStages - 1) & 1))) {
      pl.abort = true;
      eflags |= SRKV_EFLAG_TIMEOUT;
      break;
    }
    *ring.stage(s) = Int4Stage{pl.segs, 1, 0, 0, 0, 0, {0, 0}};
    mbar_arrive(ring.full(s));
    ++pl.it;
  }
  for (int64_t i = pl.it > C::kStages ? pl.it - C::kStages : 0; i < pl.it; ++i)
    if (!mbar_wait(ring.full((int)(i % C::kStages)), (uint32_t)((i / C::kStages) & 1))) {
      eflags |= SRKV_EFLAG_TIMEOUT;
      return;
    }
  for (int32_t i = pl.queries > C::kSegs ? pl.queries - C::kSegs : 0; i < pl.queries; ++i)
    if (!mbar_wait(ring.query(i % C::kSegs), (uint32_t)((i / C::kSegs) & 1))) {
      eflags |= SRKV_EFLAG_TIMEOUT;
      return;
    }
}

// The consumer warps' part (warp: 0 .. kWarps - 1).
template <int D, int Fmt>
__device__ __forceinline__ void consumer_loop_int4(const DecodeArgs& a, unsigned char* smem,
                                                   int lane, int warp) {
  constexpr bool kNarrow = Fmt == kInt4Narrow;
  using C = Cfg<D, Fmt>;
  using F = Int4Slab<D>;
  constexpr int kGroupWarps = C::kGroupWarps;       // warps per page
  constexpr int kGroups = C::kGroups;               // pages at once
  const Int4Ring<D, Fmt> ring{smem};
  constexpr int kTok = kBlock / kGroupWarps;        // tokens per warp and page
  constexpr int NW = kTok / 32;                     // 32-token groups per warp
  constexpr int KW = D / 32;                        // key words per lane and row
  constexpr int VX = D / 32;                        // 16-byte value loads per lane and octet
  constexpr int R = kNarrow ? 1 : 2;                // rows of a tile in a lane's softmax
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
  const Lane ln{lane >> 2, lane & 3};
  const int group = warp / kGroupWarps, row0 = (warp % kGroupWarps) * kTok;
  const int tile_row = 8 * (ln.g >> 1) + (ln.g & 1);  // token of tile row g within 32 tokens
  const bool second = kNarrow && ln.t >= 2;           // this lane takes rows g + 8
  const int my_row = row0 + tile_row + (second ? 2 : 0);
  const int hd = kNarrow ? 2 * (ln.t & 1) : 2 * ln.t;  // this lane's heads: hd, hd + 1
  // lanes of the same heads: the g's, and with kNarrow also t + 2
  constexpr int kFirstXor = kNarrow ? 2 : 4;
  SoftmaxState<D> st;
  st.reset();
  float pm[2] = {0.f, 0.f};  // sum of weight * vlo of the lane's heads and tokens
  // weight * vs to the fp16 operand, for each head: 2^11 over its lim (rows g + 8: 16 times less, here
  // for kNarrow, in their vs otherwise).  lim is 2^-100 at least, and that at first.
  const float vf_start = exp2_of(kInt4PLog2 + 100) * (second ? 0.0625f : 1.f);
  float vf[2] = {vf_start, vf_start};
  uint32_t qb[KW][2][2];     // [word][bits 0..7, 8..15 of its halves][codes * 2^-24, * 2^-20]
#pragma unroll
  for (int i = 0; i < KW; ++i) qb[i][0][0] = qb[i][0][1] = qb[i][1][0] = qb[i][1][1] = 0u;
  float qs0 = 0.f, qs1 = 0.f;  // factors of the lane's heads' logits (log2 domain)
  float qm0 = 0.f, qm1 = 0.f;  // sum_d q_d of the lane's heads (log2 domain)

  // Leaves this warp's state of segment `seg` for the merger (once it is done with the segment
  // before).  False: a wait ran out.
  auto leave = [&](int32_t seg) {
#pragma unroll
    for (int o = kFirstXor; o < 32; o <<= 1) {
      st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], o);
      st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], o);
      pm[0] += __shfl_xor_sync(0xffffffffu, pm[0], o);
      pm[1] += __shfl_xor_sync(0xffffffffu, pm[1], o);
    }
    // only NaN rows seen: a finite reference, so that the merges do not take the part for empty
    if (st.m[0] == -INFINITY && !(st.l[0] == 0.f)) st.m[0] = 0.f;
    if (st.m[1] == -INFINITY && !(st.l[1] == 0.f)) st.m[1] = 0.f;
    if (seg > 0 && !mbar_wait(ring.merged(), (uint32_t)((seg - 1) & 1))) return false;
    if (!kNarrow || ln.t < 2) {
      const float unit0 = exp2_of(24) * inverse_exp2(vf[0]);  // 2^24 of the subnormals
      const float unit1 = exp2_of(24) * inverse_exp2(vf[1]);
      const int slot = kNarrow ? ln.g * 2 + ln.t : lane;
      float4* p = reinterpret_cast<float4*>(
          ring.state(warp * C::kState + slot * C::kStateStride));
      p[0] = make_float4(st.m[0], st.m[1], st.l[0], st.l[1]);
#pragma unroll
      for (int i = 0; i < C::MT; ++i)
        p[1 + i] = make_float4(fmaf(st.acc[i][0], unit0, pm[0]), fmaf(st.acc[i][1], unit1, pm[1]),
                               fmaf(st.acc[i][2], unit0, pm[0]), fmaf(st.acc[i][3], unit1, pm[1]));
    }
    warp_arrive(ring.left());
    return true;
  };

  // The unit's query: fp16 with a power of two for each head, its largest magnitude put into
  // [2^14, 2^15), so that bf16's 8 significant bits stay exact down to 2^-25 of it.
  auto load_query = [&](const unsigned char* q) {
    constexpr int QV = D / 32;  // 16-byte loads: elements (D / 4) t .. of the column's head
    const int head = kNarrow ? ln.g & 3 : ln.g;
    int4 w[QV];
    uint32_t top = 0u;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < QV; ++i) {
      w[i] = head < a.G ? lds128(q + ((size_t)head * D + (D / 4) * ln.t + 8 * i) * 2)
                        : make_int4(0, 0, 0, 0);
      const uint32_t u[4] = {(uint32_t)w[i].x, (uint32_t)w[i].y, (uint32_t)w[i].z,
                             (uint32_t)w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = (u[e] << 16) & 0x7fffffffu, y = u[e] & 0x7fff0000u;
        if (x < 0x7f800000u) top = max(top, x);  // the largest finite magnitude
        if (y < 0x7f800000u) top = max(top, y);
        sum += bf16_lo(u[e]) + bf16_hi(u[e]);
      }
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    qm0 = __shfl_sync(0xffffffffu, sum, 4 * hd) * a.scale_log2;
    qm1 = __shfl_sync(0xffffffffu, sum, 4 * hd + 4) * a.scale_log2;
    int e = (int)(top >> 23) - 127;        // floor(log2 top), -127 for zeros and subnormals
    e = min(max(e, -112), 100);
    const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    const float qs = __uint_as_float((uint32_t)(127 + 10 + e) << 23) * a.scale_log2;  // 2^(24 - 14 + e)
    qs0 = __shfl_sync(0xffffffffu, qs, 4 * hd);
    qs1 = __shfl_sync(0xffffffffu, qs, 4 * hd + 4);
#pragma unroll
    for (int i = 0; i < QV; ++i) {
      const uint32_t u[4] = {(uint32_t)w[i].x, (uint32_t)w[i].y, (uint32_t)w[i].z,
                             (uint32_t)w[i].w};
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // the pair in nibble p of both halves
        const float fp = (p & 1) ? f * 0.0625f : f;
        qb[i][p >> 1][p & 1] = pack_f16(bf16_lo(u[p]) * fp, bf16_hi(u[p]) * fp);
      }
    }
  };

  // The warp's tokens of the page in stage s.
  auto attend = [&](const Int4Stage& inf, const unsigned char* slab) {
    const uint32_t* k_rows = reinterpret_cast<const uint32_t*>(slab + F::kKRows) + my_row;
    const uint32_t* v_rows = reinterpret_cast<const uint32_t*>(slab + F::kVRows) + my_row;
    // ---- logits (log2 domain) of the lane's rows and heads, and vs and vlo of the rows
    float z[NW][2][R][2], vs[NW][2][R], vl[NW][2][R];
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int ra = row0 + 32 * w + tile_row + 4 * j, rb = ra + 2;
        uint32_t ka[KW], kb[KW];
        if constexpr (KW == 4) {
          const int4 x = lds128(slab + ra * (D / 2) + ln.t * 16);
          const int4 y = lds128(slab + rb * (D / 2) + ln.t * 16);
          ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
          kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
        } else {
          const int2 x = *reinterpret_cast<const int2*>(slab + ra * (D / 2) + ln.t * 8);
          const int2 y = *reinterpret_cast<const int2*>(slab + rb * (D / 2) + ln.t * 8);
          ka[0] = x.x, ka[1] = x.y;
          kb[0] = y.x, kb[1] = y.y;
        }
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KW; ++i)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t x = ka[i] >> (8 * p), y = kb[i] >> (8 * p);
            mma_16816_f16(acc, x & kLow, y & kLow, x & kHigh, y & kHigh, qb[i][p][0], qb[i][p][1]);
          }
#pragma unroll
        for (int x = 0; x < R; ++x) {
          const uint32_t kr = k_rows[32 * w + 4 * j + 2 * x], vr = v_rows[32 * w + 4 * j + 2 * x];
          const float c0 = kNarrow ? (second ? acc[2] : acc[0]) : acc[2 * x];
          const float c1 = kNarrow ? (second ? acc[3] : acc[1]) : acc[2 * x + 1];
          const float ks = int4_scale(kr), lo = int4_lo(kr);
          z[w][j][x][0] = fmaf(c0, ks * qs0, lo * qm0);
          z[w][j][x][1] = fmaf(c1, ks * qs1, lo * qm1);
          vs[w][j][x] = int4_scale(vr) * (x == 0 ? 1.f : 0.0625f);
          vl[w][j][x] = int4_lo(vr);
        }
      }
    // ---- rows that are not attended: weight 0, and their parameters are not data
    const bool whole = inf.lo <= row0 && inf.hi >= row0 + kTok &&
                       (inf.ie >= row0 + kTok || inf.ws <= row0 || inf.ws <= inf.ie);
    if (!whole) {
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < R; ++x) {
            const int r = my_row + 32 * w + 4 * j + 2 * x;
            if (!(r >= inf.lo && r < inf.hi && (r < inf.ie || r >= inf.ws))) {
              z[w][j][x][0] = z[w][j][x][1] = -INFINITY;
              vs[w][j][x] = vl[w][j][x] = 0.f;
            }
          }
    }
    // ---- weights, and as operands of the second product times vs: fp16 (half a step is 2^-11 of
    //      each, independent over the tokens)
    float ex[NW][2][R][2];
    auto weigh = [&] {
      const float base0 = st.m[0] == -INFINITY ? 0.f : st.m[0];
      const float base1 = st.m[1] == -INFINITY ? 0.f : st.m[1];
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < R; ++x) {
            ex[w][j][x][0] = fast_exp2(z[w][j][x][0] - base0);
            ex[w][j][x][1] = fast_exp2(z[w][j][x][1] - base1);
          }
    };
    uint32_t p[NW][2][R], top;
    auto operands = [&] {
      top = 0u;
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < R; ++x) {
            const float v = vs[w][j][x];
            p[w][j][x] = pack_f16(ex[w][j][x][0] * v * vf[0], ex[w][j][x][1] * v * vf[1]);
            top = max_f16x2(top, p[w][j][x]);  // (a NaN stays)
          }
    };
    weigh();
    operands();
    // ---- raise the references if some weight or operand passes them
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int x = 0; x < R; ++x) {
          mx0 = fmaxf(mx0, z[w][j][x][0]);
          mx1 = fmaxf(mx1, z[w][j][x][1]);
        }
    const bool past = ((top + 0x08000800u) & 0x80008000u) != 0u;  // a half of 2^15 or more, or NaN
    if (__any_sync(0xffffffffu,
                   mx0 > st.m[0] + kInt4Headroom || mx1 > st.m[1] + kInt4Headroom || past)) {
#pragma unroll
      for (int o = kFirstXor; o < 32; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      const float n0 = fmaxf(st.m[0], mx0), n1 = fmaxf(st.m[1], mx1);
      const float a0 = n0 == -INFINITY ? 1.f : fast_exp2(st.m[0] - n0);
      const float a1 = n1 == -INFINITY ? 1.f : fast_exp2(st.m[1] - n1);
      st.m[0] = n0;
      st.m[1] = n1;
      st.l[0] *= a0;
      st.l[1] *= a1;
      pm[0] *= a0;
      pm[1] *= a1;
      weigh();
      float u0 = 0.f, u1 = 0.f;  // the largest weight * vs of these rows
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < R; ++x) {
            const float v = vs[w][j][x] * (x == 0 ? 1.f : 16.f);
            u0 = fmaxf(u0, ex[w][j][x][0] * v);
            u1 = fmaxf(u1, ex[w][j][x][1] * v);
          }
#pragma unroll
      for (int o = kFirstXor; o < 32; o <<= 1) {
        u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, o));
        u1 = fmaxf(u1, __shfl_xor_sync(0xffffffffu, u1, o));
      }
      // Sets f for products up to u beside accumulators of the old lim times a; returns what they are
      // multiplied by.  lim becomes the power of two above u or the one below the old lim times a, the
      // larger one, within 2^-100 .. 2^110: never more than twice the largest product met.
      auto raise = [&](float& f, float u, float a) {
        const float one = exp2_of(kInt4PLog2) * (second ? 0.0625f : 1.f);
        const float old = inverse_exp2(f) * one * a;
        const uint32_t e = min(max(max((__float_as_uint(u) >> 23) + 1u, __float_as_uint(old) >> 23),
                                   27u), 237u);
        const float inv = __uint_as_float((254u - e) << 23);
        f = inv * one;
        return old * inv;
      };
      const float g0 = raise(vf[0], u0, a0), g1 = raise(vf[1], u1, a1);
#pragma unroll
      for (int i = 0; i < C::MT; ++i) {
        st.acc[i][0] *= g0;
        st.acc[i][1] *= g1;
        st.acc[i][2] *= g0;
        st.acc[i][3] *= g1;
      }
      operands();
    }
    uint32_t b[NW][2][2];
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int x = 0; x < R; ++x) {
          const float e0 = ex[w][j][x][0], e1 = ex[w][j][x][1];
          st.l[0] += e0;
          st.l[1] += e1;
          pm[0] = fmaf(e0, vl[w][j][x], pm[0]);
          pm[1] = fmaf(e1, vl[w][j][x], pm[1]);
          p[w][j][x] = movmatrix_trans(p[w][j][x]);
        }
        b[w][j][0] = p[w][j][0];
        b[w][j][1] = kNarrow ? __shfl_xor_sync(0xffffffffu, p[w][j][0], 16) : p[w][j][R - 1];
      }
    // ---- O^T += V^T . P.  The products of this page's tokens are summed from zero and added in
    // fp32: a tensor core's sums truncate, and over a long segment of nearly equal weights that
    // drift would show against the small difference of sum u c and sum w lo that is the output.
    const unsigned char* v = slab + F::kVCodes + (row0 / 32) * (D / 4) * 64 + ln.t * 16;
#pragma unroll
    for (int x = 0; x < VX; ++x) {
      float o[2][4] = {};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int4 q4 = lds128(v + (w * (D / 4) + ln.g + 8 * x) * 64);
        const uint32_t u[4] = {(uint32_t)q4.x, (uint32_t)q4.y, (uint32_t)q4.z, (uint32_t)q4.w};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t p = u[2 * h] >> (8 * j), q = u[2 * h + 1] >> (8 * j);
            mma_16816_f16(o[h], p & kLow, q & kLow, p & kHigh, q & kHigh, b[w][j][0], b[w][j][1]);
          }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) st.acc[2 * x + h][c] += o[h][c];
    }
  };

  int s = group;  // this group's stages: group, group + kGroups, ...
  uint32_t parity = 0u;
  int32_t cur = -1;  // the segment the state belongs to
  bool ok = true;
  for (;;) {
    ok = mbar_wait(ring.full(s), parity);
    if (!ok) break;
    const Int4Stage inf = *ring.stage(s);
    while (cur < inf.seg && ok) {  // the segments up to this one are over for this warp
      if (cur >= 0) ok = leave(cur);
      ++cur;
      st.reset();
      pm[0] = pm[1] = 0.f;
      vf[0] = vf[1] = vf_start;
      if (cur == inf.seg && !inf.last && ok) {
        ok = mbar_wait(ring.query(cur % C::kSegs), (uint32_t)((cur / C::kSegs) & 1));
        load_query(ring.q(cur % C::kSegs));
      }
    }
    if (!ok || inf.last) break;
    if (row0 < inf.hi && row0 + kTok > inf.lo) attend(inf, ring.slab(s));
    warp_arrive(ring.empty(s));  // release the stage
    s += kGroups;
    if (s >= C::kStages) {
      s -= C::kStages;
      parity ^= 1u;
    }
  }
  // after the last segment is merged, tell the merger that there is no other
  if (ok && cur > 0) ok = mbar_wait(ring.merged(), (uint32_t)((cur - 1) & 1));
  if (!ok) {
    if (lane == 0) raise_flags(a.error_flags, SRKV_EFLAG_TIMEOUT);
    return;
  }
  if (lane == 0) *ring.done() = 1;
  warp_arrive(ring.left());
}

// The merger warp: segment after segment, joins the consumer warps' states and calls
// write_partial(state, segment, lane) with the result.
template <int D, int Fmt, typename WritePartial>
__device__ __forceinline__ void merger_loop_int4(const DecodeArgs& a, unsigned char* smem, int lane,
                                                 WritePartial&& write_partial) {
  using C = Cfg<D, Fmt>;
  const Int4Ring<D, Fmt> ring{smem};
  const Lane ln{lane >> 2, lane & 3};
  constexpr bool kNarrow = Fmt == kInt4Narrow;
  // Groups of at most 4 heads: lanes t and t + 2 hold the same heads and take half of the warps each.
  constexpr int kShare = kNarrow ? C::kWarps / 2 : C::kWarps;
  const int slot = kNarrow ? ln.g * 2 + (ln.t & 1) : lane;
  const float4* mine = reinterpret_cast<const float4*>(
      ring.state((kNarrow && ln.t >= 2 ? kShare : 0) * C::kState + slot * C::kStateStride));
  for (int32_t seg = 0;; ++seg) {
    if (!mbar_wait(ring.left(), (uint32_t)(seg & 1))) {
      if (lane == 0) raise_flags(a.error_flags, SRKV_EFLAG_TIMEOUT);
      return;
    }
    if (*ring.done()) return;
    SoftmaxState<D> st;
    st.reset();
    float f0[kShare], f1[kShare];  // the shares' references, then their weights
    float l0[kShare], l1[kShare];
#pragma unroll
    for (int w = 0; w < kShare; ++w) {
      const float4 ml = mine[w * (C::kState / 4)];
      f0[w] = ml.x, f1[w] = ml.y, l0[w] = ml.z, l1[w] = ml.w;
      st.m[0] = fmaxf(st.m[0], ml.x);
      st.m[1] = fmaxf(st.m[1], ml.y);
    }
    if constexpr (kNarrow) {
      st.m[0] = fmaxf(st.m[0], __shfl_xor_sync(0xffffffffu, st.m[0], 2));
      st.m[1] = fmaxf(st.m[1], __shfl_xor_sync(0xffffffffu, st.m[1], 2));
    }
    const float b0 = st.m[0] == -INFINITY ? 0.f : st.m[0];
    const float b1 = st.m[1] == -INFINITY ? 0.f : st.m[1];
#pragma unroll
    for (int w = 0; w < kShare; ++w) {
      f0[w] = fast_exp2(f0[w] - b0);
      f1[w] = fast_exp2(f1[w] - b1);
      st.l[0] = fmaf(l0[w], f0[w], st.l[0]);
      st.l[1] = fmaf(l1[w], f1[w], st.l[1]);
    }
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
      for (int w = 0; w < kShare; ++w) {
        const float4 v = mine[w * (C::kState / 4) + 1 + i];
        st.acc[i][0] = fmaf(v.x, f0[w], st.acc[i][0]);
        st.acc[i][1] = fmaf(v.y, f1[w], st.acc[i][1]);
        st.acc[i][2] = fmaf(v.z, f0[w], st.acc[i][2]);
        st.acc[i][3] = fmaf(v.w, f1[w], st.acc[i][3]);
      }
    if constexpr (kNarrow) {
      st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], 2);
      st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], 2);
#pragma unroll
      for (int i = 0; i < C::MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          st.acc[i][c] += __shfl_xor_sync(0xffffffffu, st.acc[i][c], 2);
    }
    const Int4Segment sg = *ring.segment(seg % C::kSegs);
    warp_arrive(ring.merged());
    write_partial(st, sg, ln);
  }
}

}  // namespace srkv
