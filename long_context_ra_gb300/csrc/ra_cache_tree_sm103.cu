// Attention over the paged cache for many query rows per key head (trees of
// drafts, chunks of a prompt): bf16 queries, bf16 or 8-bit cache, tcgen05.
//
// The g x T query rows of a key head are one operand: a unit is up to two
// 128-row tiles of them, and every key tile that is brought in feeds all.
// One persistent CTA per SM walks its run of key tiles (ra_paged.cuh).
//
//   S = Q K^T        tcgen05.mma, bf16 -> fp32 in TMEM
//   p = 2^(s - m)    softmax warps, thread = row, P (bf16) over S in TMEM
//   O += P V         tcgen05.mma
//
// Two streams keep the tensor cores and the exponentials busy together.
// With two query tiles (kTwo) a stream is a query tile and both share a key
// tile of 128; with one, a stream is every other key tile, with a state of its
// own, and the two states are joined at the end of the unit.  Four tiles are
// held while two streams are at work, so at d = 128 those are of 64 keys, which
// leaves room for tiles on their way; at d = 64 128 keys fit (2 sequences of
// 60000, 8 heads, 64 rows: 82 -> 61 us, out of 8 bits 99 -> 80; 58 and 78 with
// the later steps).
//
// Over stretches (ra_cache_attention_shared) a unit's rows come from several
// sequences: the query warp gathers them row by row (tile::gather4).
//
// Warp roles (640 threads, 96 registers each at launch; the wide form below has
// 384 of 168):
//   warps 0-3, 4-7   softmax of stream 0, 1                            (112)
//   warp  9          loader: TMA boxes of the key and value tiles      (112)
//   warp  10         TMA boxes of the queries
//   warp  11         TMEM allocator, MMA issuer: the warp walks along as a whole
//                    and one lane issues, so that its operands stay in uniform
//                    registers (24 trees of 32 over 65536: 1087 -> 799 us, with
//                    a shared context 553 -> 501)
//   warps 12-19      8-bit cache: conversion, two tiles under way       (72)
//   (bf16 cache)     warp 12: tiles that end a sequence
// 3 x 128 x 112 + 2 x 128 x 72 = 61440 = 640 x 96.
//
// A tile is a row of pages: the loader's lanes look up a page each, one tile
// ahead, and bring it as one TMA box of a [pages x heads, page, d] view; a
// page that does not exist is a box behind the view, which TMA fills with
// zeros.  bf16 tiles land as operands.  Only value tiles that hold drafts or
// the end of the sequence pass through warp 12, which clears the rows behind
// the end.  8-bit tiles land in a raw ring and become bf16 in warps 12-19,
// with the row's scale inside: code * 2^e has 4 significant bits, so it is
// exact in bf16 for values above 2^-126, and neither the scores nor the
// probabilities need to know the scale.
//
// Code size sets the pace before anything else: 20 warps in five roles share
// one instruction cache.  With the score and exponential loops unrolled a tile
// of 128 keys and 256 rows took 7.3 us; rolled, 3.  (Where nothing is converted and
// two tiles of rows are at work, over stretches, the wide form has 12 warps, and
// softmax threads of 200 registers that hold a row's 128 scores of a tile: one
// pass over TMEM, not two.)  Every role is a short loop
// in 32-bit arithmetic with the unit's constants taken out: a role of one warp
// that spends some hundred instructions on an item is slower than the 1.1 us
// of tensor time that the tile needs.
//
// Measured per tile of 128 keys on one SM (152 at work, d = 128): one query
// tile, bf16 1.4 us (the tile's bytes alone take 1.5 at the copy rate), 8 bits
// 2.0; two query tiles, bf16 1.7 us, wide 1.2 (the products alone 1.1), 8 bits
// 2.2.  d = 64: 0.7, 1.1; 1.4, 1.6.
// 488 rows over 2^20 keys of 8 heads out of 8 bits: 1.88 ms, 59 % of the tensor
// rate.  A unit costs some 8 us beside its tiles: pipeline start (clocks from
// the launch: place in the division 2900, queries and first keys 6200, scores
// 7900, probabilities 10400, first results 12300) and end (5000 for 256 rows'
// parts).  So the queries come by TMA from a warp of their own, the next unit's
// as soon as the last scores of the present one are out (by 224 threads they
// were there at 9700), and results leave in whole lines (12100 by rows).
//
// Unseen drafts: their scores are -inf, so p = 0; value rows of drafts are
// looked through for elements that are not finite.  Those become 0 in the
// operand, and a unit that met one adds them at its end, row by row, to the
// queries that see them.  Rows of the context, which every query sees, stay
// as they are.
//
// Every wait is bounded, as in the forward kernel.

#include "ra_cache_attn.cuh"
#include "sm103_pipeline.cuh"
#include "sm103_ptx.cuh"

namespace ra {
namespace {

using namespace ptx;
using namespace sm103;

// kWide: nothing is converted, and the softmax warps hold a row's scores of a
// tile in registers.
template <bool kWide>
struct Roles {
  static constexpr int kThreads = kWide ? 384 : 640;
  static constexpr uint32_t kRegs = kWide ? 168 : 96;       // per thread at launch
  static constexpr uint32_t kRegsSoftmax = kWide ? 200 : 112;
  static constexpr uint32_t kRegsMain = kWide ? 104 : 112;   // MMA issuer, loader
  static constexpr uint32_t kRegsHand = kWide ? 104 : 72;    // queries, conversion
  static constexpr int kLoadWarp = kWide ? 8 : 9;
  static constexpr int kQueryWarp = 10;
  static constexpr int kMmaWarp = kWide ? 9 : 11;
  static constexpr int kHandWarp = kWide ? 11 : 12;
  static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsMain + (kWide ? 0 : 2 * 128 * kRegsHand) == kThreads * kRegs,
                "register split must equal the launch's register total");
};
constexpr uint32_t kTmemCols = 512;
// Stretches: how far above the largest score the reference is put when it moves.
// Any reference gives the same l and o; one that moves costs the tile's softmax
// a pass over O, and the largest of some 10^4 scores is further above that of a
// first tile than kRescaleLog2 where key rows are of unlike length.
constexpr float kHeadroom = 16.0f;

template <bool k8, int D, bool kTwo>
struct Layout {
  static constexpr int kKeys = kTwo || D == 64 ? 128 : 64;  // per tile
  static constexpr int kQBox = 128 * 128;        // 128 rows x 128 bytes (64 bf16)
  static constexpr int kBox = kKeys * 128;
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kTile = kKeys * D * 2;
  static constexpr int kRawTile = kKeys * D;
  static constexpr int kStages = kTwo ? (D == 128 ? (k8 ? 3 : 5) : (k8 ? 5 : 8))
                                      : (D == 128 ? (k8 ? 6 : 9) : (k8 ? 6 : 9));
  static constexpr int kRawStages = !k8 ? 0 : kTwo ? (D == 128 ? 4 : 8) : (D == 128 ? 6 : 8);
  static constexpr int kTeam = 128;  // threads that convert a tile
  static constexpr int kLoadStages = k8 ? kRawStages : kStages;  // of the ring the loader fills
  // the second query tile, or the exchange of the two streams' states: per
  // stream [128][33] floats, and [128][2]
  static constexpr int kSecond = kTwo ? kQTile : 36 * 1024;
  static constexpr int kQ0 = 0;
  static constexpr int kQ1 = kQTile;
  static constexpr int kKV = kQTile + kSecond;
  static constexpr int kRaw = kKV + kStages * kTile;
  static constexpr int kRawExp = kRaw + kRawStages * kRawTile;
  static constexpr int kBar = kRawExp + kRawStages * kKeys;
  static constexpr int kNumBars = 2 + 2 * kStages + 12 + kLoadStages + kRawStages;
  static constexpr int kMisc = (kBar + kNumBars * 8 + 15) / 16 * 16;  // TMEM base, abort flag
  // Rings of the last 32 units and key tiles: the loader is at most
  // kLoadStages + kStages <= 24 items (12 key tiles, 12 units) ahead.
  static constexpr int kPoison = kMisc + 16;        // [32]
  static constexpr int kLeftOut = kPoison + 128;    // [32]
  static constexpr int kDivision = kLeftOut + 128;
  // walks of the 8 softmax warps: in shared memory, not in registers
  static constexpr int kWalks = (kDivision + static_cast<int>(sizeof(DivisionShared)) + 15) / 16 * 16;
  static constexpr int kBytes = kWalks + 8 * static_cast<int>(sizeof(StretchWalk));  // the larger of the two
  static constexpr int kSmem = kBytes + 1024;  // slack for 1024-byte alignment
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kRawStages + kStages <= 24, "rings");
};

template <typename L>
struct Bars {
  static constexpr int kS = L::kStages;
  uint32_t base;
  __device__ uint32_t q_full() const { return base; }
  __device__ uint32_t q_empty() const { return base + 8; }
  __device__ uint32_t kv_full(int s) const { return base + 8 * (2 + s); }
  __device__ uint32_t kv_empty(int s) const { return base + 8 * (2 + kS + s); }
  __device__ uint32_t s_full(int t) const { return base + 8 * (2 + 2 * kS + t); }
  __device__ uint32_t p_full(int t) const { return base + 8 * (4 + 2 * kS + t); }
  __device__ uint32_t o_full(int t) const { return base + 8 * (6 + 2 * kS + t); }
  __device__ uint32_t x_full(int i) const { return base + 8 * (8 + 2 * kS + i); }
  __device__ uint32_t x_empty(int i) const { return base + 8 * (10 + 2 * kS + i); }
  __device__ uint32_t drain() const { return base + 8 * (12 + 2 * kS); }
  __device__ uint32_t q_raw() const { return base + 8 * (13 + 2 * kS); }
  __device__ uint32_t raw_full(int s) const { return base + 8 * (14 + 2 * kS + s); }
  __device__ uint32_t raw_empty(int s) const { return base + 8 * (14 + 2 * kS + L::kLoadStages + s); }
};

// Position in a ring of stages.
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  template <int kStages>
  __device__ void step() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// The MMA thread takes a unit's tiles in the order K0 V0 K1 V1 ... (two query
// tiles) or K0 K1 V0 K2 V1 ... (one: two key tiles under way).  Place of V
// tile `tile` of n in that order:
template <bool kTwo>
__device__ __forceinline__ int value_item(int tile, int n) {
  return kTwo ? 2 * tile + 1 : tile + 1 == n ? 2 * n - 1 : 2 * tile + 2;
}
// f(tile, v) for the items of a unit of n tiles, in order, until f is false.
// v is a constant at each place f stands: without the tests that only value
// tiles need, key tiles are converted a tenth faster.
template <bool kTwo, typename F>
__device__ __forceinline__ bool each_item(int n, F f) {
  if (!kTwo && !f(0, false)) return false;
  for (int j = 0; j < n; ++j) {
    const int k = kTwo ? j : j + 1;
    if (k < n && !f(k, false)) return false;
    if (!f(j, true)) return false;
  }
  return true;
}

// Row (of a group's kRows) of a thread's x-th 16-byte piece of an 8-bit tile;
// 8 threads share a group.  Lanes 4-7 take the rows in another order, so that
// the 16-byte writes of a group's widened pieces meet no bank twice.
template <int D, int kRows>
__device__ __forceinline__ int piece_row(int x, int pc) {
  return D == 128 ? x ^ (pc / 4) : (pc / 4) * (kRows / 2) + (x ^ (pc / 4));
}

// One arrival on `bar` when this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Halves that are not finite bf16 values, as 0xffff masks.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return ((x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// 16 e4m3 codes times 2^(e - 127) as bf16, in the order 0 2 1 3 of every four
// (the bytes stay in their halves; queries and results follow that order).
// Sign and 7 bits moved to where bf16 has them mean value * 2^-120, so the
// factor is 2^(e - 7).  That factor passes bf16's range above e = 134, and a
// NaN code would come out as 480: both are rare and go through widen_rare.
__device__ __noinline__ uint4 widen_rare(uint2 w, uint32_t e) {
  const uint32_t f1 = min(e + 120u, 254u);
  const uint32_t up = (f1 << 7) * 0x10001u, up2 = ((e + 247u - f1) << 7) * 0x10001u;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = (i & 1) ? (i < 2 ? w.x : w.y) : (i < 2 ? w.x : w.y) << 8;  // in the high bytes
    uint32_t m = mul_bf16x2(mul_bf16x2((x >> 4) & 0x07f007f0u, up), up2);
    m |= ((x & 0x7f00u) == 0x7f00u ? 0x7fffu : 0u) |
         ((x & 0x7f000000u) == 0x7f000000u ? 0x7fff0000u : 0u);
    o[i] = m | (x & 0x80008000u);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void widen16(const uint4& w4, uint32_t e, uint32_t (&o)[8]) {
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
  uint32_t nan = 0;
#pragma unroll
  for (int z = 0; z < 4; ++z) nan |= (w[z] & 0x7f7f7f7fu) + 0x01010101u;
  if ((nan & 0x80808080u) == 0u && e <= 134u) {
    const uint32_t up = e * 0x00800080u + 120u * 0x00800080u;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      o[2 * z] = mul_bf16x2((w[z] << 4) & 0x07f007f0u, up) | ((w[z] << 8) & 0x80008000u);
      o[2 * z + 1] = mul_bf16x2((w[z] >> 4) & 0x07f007f0u, up) | (w[z] & 0x80008000u);
    }
  } else {
    const uint4 lo = widen_rare(make_uint2(w[0], w[1]), e), hi = widen_rare(make_uint2(w[2], w[3]), e);
    o[0] = lo.x, o[1] = lo.y, o[2] = lo.z, o[3] = lo.w;
    o[4] = hi.x, o[5] = hi.y, o[6] = hi.z, o[7] = hi.w;
  }
}

template <int D, int kKeys>
__device__ __forceinline__ void issue_qk(bool leader, uint32_t d_tmem, uint64_t dq, uint64_t dk) {
  if (!leader) return;
  constexpr uint32_t idesc = idesc_bf16_f32(kBM, kKeys, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    mma_bf16_ss(d_tmem, dq + desc_step((kk / 4) * (kBM * 128) + (kk % 4) * 32),
                dk + desc_step((kk / 4) * (kKeys * 128) + (kk % 4) * 32), idesc, kk > 0 ? 1u : 0u);
}

template <int D, int kKeys>
__device__ __forceinline__ void issue_pv(bool leader, uint32_t d_tmem, uint32_t p_tmem, uint64_t dv,
                                         uint32_t accumulate) {
  if (!leader) return;
  constexpr uint32_t idesc = idesc_bf16_f32(kBM, D, true);
  mma_bf16_ts(d_tmem, p_tmem, dv, idesc, accumulate);
#pragma unroll
  for (int kk = 1; kk < kKeys / 16; ++kk)
    mma_bf16_ts(d_tmem, p_tmem + kk * 8, dv + desc_step(kk * 16 * 128), idesc, 1u);
}

// p = 2^(s * scale + neg) of 32 scores as bf16 pairs at tP; adds p to acc.
__device__ __forceinline__ void exp_part(const uint32_t (&s)[32], uint64_t scale2, uint64_t neg2,
                                         uint64_t (&acc)[2], uint32_t tP) {
  uint32_t pk[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint64_t x =
        fma_f32x2(pack_f32x2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), scale2, neg2);
    float x0, x1;
    unpack_f32x2(x, x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    acc[j & 1] = add_f32x2(acc[j & 1], pack_f32x2(p0, p1));
    pk[j] = pack_bf16x2(p0, p1);
  }
  tmem_st16(tP, pk);
}

// Which of the keys pos .. pos + 31 query t sees; `left` has a bit for every
// 8 of them that are not in the cache.
__device__ __forceinline__ uint32_t first_bits(int64_t n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}
__device__ __noinline__ uint32_t seen_word(const CacheAttnArgs& a, const SeqInfo& s, int b, int t,
                                              int64_t pos, uint32_t left) {
  if (t >= s.cnt) return 0u;
  const int64_t j0 = pos - s.len;  // draft of bit 0
  uint32_t seen = first_bits(-j0);
  if (!a.mask) {
    seen = first_bits(t - j0 + 1);
  } else if (j0 > -32 && j0 < s.cnt) {
    const uint8_t* m = a.mask + b * a.mask_stride + static_cast<int64_t>(t) * a.c.T + j0;
    const int from = static_cast<int>(max(-j0, int64_t{0}));
    const int to = static_cast<int>(min(s.cnt - j0, int64_t{32}));
#pragma unroll
    for (int x = 0; x < 32; ++x)  // all loads under way together
      if (x >= from && x < to) seen |= (m[x] != 0 ? 1u : 0u) << x;
  }
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if ((left >> x) & 1u) seen &= ~(0xffu << (8 * x));
  return seen;
}

// Which of columns x .. x + 31 of the drafts that query t sees in the walk's
// part hold a value that is not finite (a bit each).
template <bool k8, int D, typename A, typename W>
__device__ __noinline__ uint32_t poisoned_columns(const A& a, const W& u, int b, int head,
                                                  int t, int x, int tile) {
  const auto& c = paged(a);
  uint32_t bad = 0;
  const int64_t end = min(u.last * tile, u.seq.keys());
  for (int64_t pos = max(u.first * tile, u.seq.len); pos < end; ++pos) {
    if (!sees(a, u.seq, b, t, pos)) continue;
    int64_t row = cache_row(c, u.b, pos);
    if (row < 0) continue;
    row += static_cast<int64_t>(head) << c.page_shift;
#pragma unroll 1
    for (int e = 0; e < 32; ++e) {
      uint32_t y;
      if (k8)
        y = widen_rare(make_uint2(static_cast<const uint8_t*>(c.v)[row * D + x + e], 0u), c.ve[row]).x;
      else
        y = static_cast<const uint16_t*>(c.v)[row * D + x + e];
      if ((y & 0x7f80u) == 0x7f80u) bad |= 1u << e;
    }
  }
  return bad;
}

// Lane 4 i + j gives y[k] to lane 4 i + k and gets that lane's y[j]: rows of a
// quad of lanes become columns, so that its lanes store neighbouring pieces.  A
// store instruction then meets 8 lines, not 32: a unit's end is bound by those.
__device__ __forceinline__ void transpose4(uint4 (&y)[4], int lane) {
#pragma unroll
  for (int z = 1; z < 4; z <<= 1) {
    const bool up = lane & z;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & z) continue;
      uint4& lo = y[k];
      uint4& hi = y[k | z];
      const uint4 give = up ? lo : hi;
      uint4 got;
      got.x = __shfl_xor_sync(0xffffffffu, give.x, z);
      got.y = __shfl_xor_sync(0xffffffffu, give.y, z);
      got.z = __shfl_xor_sync(0xffffffffu, give.z, z);
      got.w = __shfl_xor_sync(0xffffffffu, give.w, z);
      if (up)
        lo = got;
      else
        hi = got;
    }
  }
}

// What a role needs of the present unit.
struct Unit {
  int head;
  int64_t r0;  // first query row of the unit within its key head
  int64_t q0;  // its row in q, out, lse
  template <typename W>
  __device__ Unit(const CacheAttnArgs& a, const AttnPlan& p, const W& u, int64_t rows) {
    head = u.unit / p.row_tiles;
    r0 = static_cast<int64_t>(u.unit % p.row_tiles) * p.rows;
    q0 = (static_cast<int64_t>(u.b) * a.c.heads + head) * rows + r0;
  }
};

// What a softmax thread's row is.
struct RowFacts {
  int tok, b;   // its token and sequence
  int64_t q;    // its place in q (stretches)
  SeqInfo seq;  // context and new tokens that it may see
  bool exists;
};

// The tiles of a unit in the wide form's softmax: a thread holds its row's 128
// scores in registers.  A function of its own, so that what the unit's end needs
// is saved once, not in the loop: local memory there takes the products'
// bandwidth to shared memory (24 samples' trees of 32 over 65536 tokens: 501 us with
// two passes over TMEM, 448 here; in the softmax role itself a tile took 4020
// clocks, 3360 with two passes).
struct WideTiles {
  uint32_t s_full, p_full, tS, tO;
  int n, border, kt;
  uint32_t ns;
  bool warp_live;
};
template <int D, typename A, typename W>
__device__ __noinline__ float2 wide_tiles(const A& a, const W& u, const WideTiles w, const Abort ab,
                                          const uint8_t* left_out, int row, int keys) {
  float m_ref = -INFINITY, l = 0.f;
  const float scale = a.scale_log2;
  const uint64_t scale2 = pack_f32x2(scale, scale);
  uint32_t phase = w.ns;
#pragma unroll 1
  for (int it = 0; it < w.n; ++it) {
    if (!wait_warp(w.s_full, phase++ & 1u, ab)) break;
    tc_fence_after();
    if (w.warp_live) {
      const uint32_t left = *reinterpret_cast<const volatile uint32_t*>(left_out + ((w.kt + it) & 31) * 4);
      if (it >= w.border || left != 0u) {  // scores that are not seen become -inf in TMEM
        const Stretch st = paged(a).list[u.b];
        const MemberRow r(a, st, u.unit, row);
#pragma unroll 1
        for (int x = 0; x < kBN / 32; ++x) {
          const uint32_t seen = seen_word(a, SeqInfo{u.seq.len, r.cnt}, r.b, r.t, (u.first + it) * keys + 32 * x,
                                          left >> (4 * x));
          uint32_t y[32];
          __syncwarp();
          tmem_ld32(w.tS + 32 * x, y);
          tmem_ld_wait();
          reg_fence(y, 32);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((seen >> e) & 1u)) y[e] = __float_as_uint(-INFINITY);
          tmem_st32(w.tS + 32 * x, y);
        }
        tmem_st_wait();
      }
      uint32_t s[kBN];
#pragma unroll
      for (int x = 0; x < kBN; x += 32) tmem_ld32(w.tS + x, s + x);
      tmem_ld_wait();
      reg_fence(s, kBN);
      float m_new = row_max(s) * scale;
      const bool need = m_new > m_ref + kRescaleLog2;
      if (__any_sync(0xffffffffu, need)) {
        m_new += kHeadroom;
        const float alpha = need ? ex2(m_ref - m_new) : 1.f;
        if (it > 0) {
#pragma unroll 1
          for (int x = 0; x < D; x += 16) {
            uint32_t o[16];
            tmem_ld16(w.tO + x, o);
            tmem_ld_wait();
            reg_fence(o, 16);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(w.tO + x, o);
          }
          tmem_st_wait();
        }
        if (need) {
          l *= alpha;
          m_ref = m_new;
        }
      }
      const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
      l += exp_store(s, scale2, pack_f32x2(neg, neg), w.tS);
      tmem_st_wait();
    }
    tc_fence_before();
    mbar_arrive(w.p_full);
  }
  return make_float2(m_ref, l);
}

// Whether a unit has rows in its second tile.
__device__ __forceinline__ bool second_tile(const CacheAttnArgs& a, const AttnPlan& p, const UnitWalk& u,
                                            int64_t rows) {
  return Unit(a, p, u, rows).r0 + 128 < rows;
}
__device__ __forceinline__ bool second_tile(const SharedAttnArgs& a, const AttnPlan&, const StretchWalk& u, int64_t) {
  return a.stretches.list[u.b].rows > 128;
}

// The form of a launch: over stretches of two tiles of rows the wide one.
template <bool k8, bool kTwo, typename A>
struct Form {
  static constexpr bool kWide = !k8 && kTwo && IsShared<A>::value;
};
template <uint32_t kFrom, uint32_t kTo>
__device__ __forceinline__ void set_registers() {
  if constexpr (kTo > kFrom)
    setmaxnreg_inc<kTo>();
  else
    setmaxnreg_dec<kTo>();
}

template <bool k8, int D, bool kTwo, typename A>
__global__ void __launch_bounds__(Roles<Form<k8, kTwo, A>::kWide>::kThreads, 1)
    cache_tree_kernel(const __grid_constant__ A a, const __grid_constant__ AttnPlan p,
                      const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      const __grid_constant__ CUtensorMap tq) {
  using L = Layout<k8, D, kTwo>;
  constexpr bool kShared = IsShared<A>::value;
  using Walk = typename IsShared<A>::Walk;
  constexpr bool kWide = Form<k8, kTwo, A>::kWide;
  using Ro = Roles<kWide>;
  constexpr int kMmaWarp = Ro::kMmaWarp, kQueryWarp = Ro::kQueryWarp, kLoadWarp = Ro::kLoadWarp,
                kHandWarp = Ro::kHandWarp;
  constexpr int kS = L::kStages, kKeys = L::kKeys, kN = kKeys / 32;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const Bars<L> bars{base + L::kBar};
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(gbase + L::kMisc);
  const Abort ab{tmem_holder + 1, a.c.status, a.wait_limit > 0 ? a.wait_limit : kWaitLimit};
  volatile uint32_t* poison = reinterpret_cast<volatile uint32_t*>(gbase + L::kPoison);
  DivisionShared& sh = *reinterpret_cast<DivisionShared*>(gbase + L::kDivision);
  const auto& c = paged(a);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t rows = head_rows(a);

  // ---- set-up
  allow_join();
  if (threadIdx.x == 0) {
    mbar_init(bars.q_full(), k8 ? 256 : 1);
    mbar_init(bars.q_raw(), 1);
    mbar_init(bars.q_empty(), 1);
    for (int s = 0; s < kS; ++s) {
      mbar_init(bars.kv_full(s), k8 ? L::kTeam : 1);
      mbar_init(bars.kv_empty(s), 1);
    }
    for (int s = 0; s < L::kLoadStages; ++s) mbar_init(bars.raw_full(s), k8 ? 33 : 1);
    for (int s = 0; s < L::kRawStages; ++s) mbar_init(bars.raw_empty(s), L::kTeam);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bars.s_full(t), 1);
      mbar_init(bars.p_full(t), 128);
      mbar_init(bars.o_full(t), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.x_full(i), 128);
      mbar_init(bars.x_empty(i), 128);
    }
    mbar_init(bars.drain(), 1);
    *ab.flag = 0u;
    for (int i = 0; i < 32; ++i) poison[i] = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(base + L::kMisc, kTmemCols);
    tmem_relinquish();
  }
  const int64_t run = division_start(c, p.div, blockIdx.x, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp >= kHandWarp) {
    // ================= queries, conversion =================
    set_registers<Ro::kRegs, Ro::kRegsHand>();
    const int tid = threadIdx.x - kHandWarp * 32;
    // The unit's queries, in the order of widen16: in place, a piece stays in
    // its thread.
    auto order_queries = [&](const Walk& w, uint32_t ord) {
      const uint32_t end = base + L::kQ0 + (kTwo && second_tile(a, p, w, rows) ? 2 : 1) * L::kQTile;
      if (!wait_warp(bars.q_raw(), ord & 1u, ab)) return false;
#pragma unroll 1
      for (uint32_t at = base + L::kQ0 + tid * 16; at < end; at += 4 * 256 * 16) {
        uint4 q[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) q[x] = lds128(at + x * 256 * 16);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          st_shared_v4(at + x * 256 * 16, __byte_perm(q[x].x, q[x].y, 0x5410),
                       __byte_perm(q[x].x, q[x].y, 0x7632), __byte_perm(q[x].z, q[x].w, 0x5410),
                       __byte_perm(q[x].z, q[x].w, 0x7632));
      }
      fence_proxy_async_smem();
      mbar_arrive(bars.q_full());
      return true;
    };
    static_assert(!k8 || L::kQTile % (4 * 256 * 16) == 0, "whole rounds of the queries");
    Walk w;
    w.start_found(c, p.div, sh, run);
    if (k8) {
      Ring in, out;  // raw stages; operand stages
      constexpr int kTeams = 256 / L::kTeam;
      constexpr int kGroup = kKeys / (L::kTeam / 8);  // rows per 8 threads
      constexpr int kPieces = D * kKeys / 16 / L::kTeam;
      const int team = tid / L::kTeam, grp = tid % L::kTeam / 8, pc = tid % 8;
      int turn = 0;  // of the team that takes the next tile
      const uint32_t src0 = base + L::kRaw + (D == 128 ? pc : pc % 4) * 16;
      const uint32_t dst0 = base + L::kKV + (D == 128 ? pc / 4 : 0) * L::kBox;
      const int ch = 2 * (pc % 4);
      for (uint32_t ord = 0; !w.done(); ++ord, w.next(c, p.div)) {
        if (!order_queries(w, ord)) break;
        const int n = static_cast<int>(w.last - w.first);
        // keys and context keys of this part
        const int64_t before = w.first * kKeys;
        const uint32_t keys = static_cast<uint32_t>(min(w.seq.keys() - before, static_cast<int64_t>(n) * kKeys));
        const uint32_t context = static_cast<uint32_t>(
            min(max(w.seq.len - before, int64_t{0}), static_cast<int64_t>(n) * kKeys));
        const bool ok = each_item<kTwo>(n, [&](int tile, bool v) {
          const bool other = turn != team;
          turn = turn + 1 == kTeams ? 0 : turn + 1;
          if (other) {
            in.step<L::kLoadStages>();
            out.step<kS>();
            return true;
          }
          if (!wait_warp(bars.raw_full(in.stage), in.phase, ab)) return false;
          if (!wait_warp(bars.kv_empty(out.stage), out.phase ^ 1u, ab)) return false;
          const uint32_t src = src0 + in.stage * L::kRawTile;
          const uint8_t* ex = gbase + L::kRawExp + in.stage * kKeys;
          const uint32_t dst = dst0 + out.stage * L::kTile;
          const uint32_t row0 = static_cast<uint32_t>(tile) * kKeys;
          const bool border = v && row0 + kKeys > context;
          bool bad = false;
          // loads in flight; four spill, and are slower
          constexpr int kBatch = kPieces < 2 ? kPieces : 2;
#pragma unroll 1
          for (int z0 = 0; z0 < kPieces; z0 += kBatch) {
            uint4 w4[kBatch];
            uint32_t e[kBatch];
#pragma unroll
            for (int z = 0; z < kBatch; ++z) {
              const int r = grp * kGroup + piece_row<D, kGroup>(z0 + z, pc);
              w4[z] = lds128(src + r * D);
              e[z] = ex[r];
            }
#pragma unroll
            for (int z = 0; z < kBatch; ++z) {
              const int r = grp * kGroup + piece_row<D, kGroup>(z0 + z, pc);
              uint32_t o[8];
              widen16(w4[z], e[z], o);
              if (border && row0 + r >= context) {
                const bool real = row0 + r < keys;
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                  const uint32_t nf = real ? not_finite(o[y]) : 0u;
                  bad = bad || nf;
                  o[y] = real ? o[y] & ~nf : 0u;
                }
              }
              st_shared_v4(dst + r * 128 + ((ch ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
              st_shared_v4(dst + r * 128 + (((ch + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
            }
          }
          mbar_arrive(bars.raw_empty(in.stage));
          if (bad) poison[ord & 31] = ord + 1u;
          fence_proxy_async_smem();
          mbar_arrive(bars.kv_full(out.stage));
          in.step<L::kLoadStages>();
          out.step<kS>();
          return true;
        });
        if (!ok) break;
      }
    } else if (warp == kHandWarp) {
      // value tiles with drafts or the end
      uint32_t first_item = 0, used = 0;  // items before the unit; phases of raw_full, a bit each
      bool ok = true;
      for (uint32_t ord = 0; ok && !w.done(); ++ord, w.next(c, p.div)) {
        const int n = static_cast<int>(w.last - w.first);
        const int64_t before = w.first * kKeys;
        const uint32_t keys = static_cast<uint32_t>(min(w.seq.keys() - before, static_cast<int64_t>(n) * kKeys));
        const uint32_t context = static_cast<uint32_t>(
            min(max(w.seq.len - before, int64_t{0}), static_cast<int64_t>(n) * kKeys));
        const int from =
            static_cast<int>(min(max(w.seq.len / kKeys - w.first, int64_t{0}), static_cast<int64_t>(n)));
        for (int tile = from; tile < n; ++tile) {
          const int stage = static_cast<int>((first_item + value_item<kTwo>(tile, n)) % kS);
          if (!wait_warp(bars.raw_full(stage), (used >> stage) & 1u, ab)) {
            ok = false;
            break;
          }
          used ^= 1u << stage;
          bool bad = false;
          // the rows behind the context, 16-byte pieces, four at a time
          const uint32_t at = base + L::kKV + stage * L::kTile + (lane % 8) * 16;
          const uint32_t row0 = static_cast<uint32_t>(tile) * kKeys;
          const int skip = context > row0 ? static_cast<int>(context - row0) : 0;
          constexpr int kBoxes = D / 64;
#pragma unroll 1
          for (int i0 = skip + lane / 8; i0 < kKeys; i0 += 16 / kBoxes) {
            uint4 y[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int r = i0 + 4 * (z / kBoxes);
              y[z] = r < kKeys ? lds128(at + (z % kBoxes) * L::kBox + r * 128) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int r = i0 + 4 * (z / kBoxes);
              const uint32_t n0 = not_finite(y[z].x), n1 = not_finite(y[z].y), n2 = not_finite(y[z].z),
                             n3 = not_finite(y[z].w);
              if (r >= kKeys) continue;
              const uint32_t to = at + (z % kBoxes) * L::kBox + r * 128;
              if (row0 + r >= keys) {
                st_shared_v4(to, 0u, 0u, 0u, 0u);
              } else if (n0 | n1 | n2 | n3) {
                bad = true;
                st_shared_v4(to, y[z].x & ~n0, y[z].y & ~n1, y[z].z & ~n2, y[z].w & ~n3);
              }
            }
          }
          if (bad) poison[ord & 31] = ord + 1u;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.kv_full(stage));
        }
        first_item += 2u * static_cast<uint32_t>(n);
      }
    }
  } else if (warp == kLoadWarp) {
    // ================= loader =================
    set_registers<Ro::kRegs, Ro::kRegsMain>();
    const int page_rows = min(1 << c.page_shift, kKeys);  // of a box
    const int boxes = kKeys / page_rows;
    constexpr int kHalves = k8 ? 1 : D / 64;
    const bool mine = lane < boxes * kHalves;
    const int box = lane % boxes, half = lane / boxes;
    const uint32_t dst_off =
        half * L::kBox + box * page_rows * (k8 ? D : 128) + (k8 ? L::kRaw : L::kKV) + base;
    constexpr uint32_t kLoadTile = k8 ? L::kRawTile : L::kTile;
    const int from = min(lane * 8 / page_rows, boxes - 1);  // the box of rows 8 lane ..
    const uint32_t in_page = (1u << c.page_shift) - 1u;
    const int32_t behind = static_cast<int32_t>((c.pages > 0 ? c.pages * c.heads : 1));
    const uint64_t map_k = reinterpret_cast<uint64_t>(&tk), map_v = reinterpret_cast<uint64_t>(&tv);
    Walk w;
    w.start_found(c, p.div, sh, run);
    Ring r;
    uint32_t ktiles = 0;
    // a bit per stage: loaded, to arrive at raw_full, and the phase of that
    uint32_t issued = 0, hand = 0, last = 0, raw_phase = 0;
    bool ok = static_cast<int64_t>(blockIdx.x) != a.stall_cta;
    for (; ok && !w.done(); w.next(c, p.div)) {
      const int n = static_cast<int>(w.last - w.first);
      const int head = w.unit / p.row_tiles;
      const uint32_t pos0 = static_cast<uint32_t>(w.first) * kKeys;  // positions stay below 2^32
      const uint32_t keys = static_cast<uint32_t>(w.seq.keys());
      // the first tile with drafts or the end
      const int border =
          static_cast<int>(min(max(w.seq.len / kKeys - w.first, int64_t{0}), static_cast<int64_t>(n)));
      const int32_t* row_of_table = pages_of(c, w.b);
      const uint32_t columns = static_cast<uint32_t>(columns_of(c, w.b));
      // this lane's page of a tile: its number, -1 for one that is missing,
      // -2 for none
      auto look_up = [&](int tile) {
        const uint32_t pos = pos0 + static_cast<uint32_t>(tile) * kKeys + box * page_rows;
        if (!mine || tile >= n || pos >= keys) return -2;
        const uint32_t col = pos >> c.page_shift;
        return col < columns ? max(__ldg(row_of_table + col), -1) : -1;
      };
      int page = -2, ahead = look_up(0);  // of the last key tile loaded; of the next
      int32_t z = 0, zv = 0;              // its TMA coordinate; that of the value tile to come
      int64_t erow = 0, erow_v = 0;       // exponent rows (8 per lane), -1: none
      ok = each_item<kTwo>(n, [&](int tile, bool v) {
        if (!v) {
          page = ahead;
          ahead = look_up(tile + 1);
          const bool there = page >= 0 && page < c.pages;
          const uint32_t lost = __ballot_sync(0xffffffffu, page != -2 && !there);
          uint32_t left = 0;  // bit i: rows 8 i .. 8 i + 7 are wanted but not in the cache
          if (lost) {
            if (page != -2 && !there) flag_page(c.status);
            left = __ballot_sync(0xffffffffu, lane < kKeys / 8 && ((lost >> from) & 1u));
          }
          if (lane == 0)
            *reinterpret_cast<volatile uint32_t*>(gbase + L::kLeftOut + (ktiles & 31u) * 4) = left;
          ++ktiles;
          zv = z;
          z = there ? page * c.heads + head : behind;
          if (k8) {
            erow_v = erow;
            const int32_t ze = __shfl_sync(0xffffffffu, z, from);
            const uint32_t pos = pos0 + static_cast<uint32_t>(tile) * kKeys + lane * 8;
            erow = lane < kKeys / 8 && ze != behind
                       ? (static_cast<int64_t>(ze) << c.page_shift) + (pos & in_page)
                       : -1;
          }
        }
        // in the order with two key tiles under way the value tile is the one
        // before, unless it is the last
        const bool older = !kTwo && v && tile + 1 < n;
        const int32_t zz = older ? zv : z;
        if (!wait_warp(k8 ? bars.raw_empty(r.stage) : bars.kv_empty(r.stage), r.phase ^ 1u, ab))
          return false;
        // where the arrival is seen: by the MMA thread, or by who converts or clears
        const bool by_hand = k8 || (v && tile >= border);
        const uint32_t bar = by_hand ? bars.raw_full(r.stage) : bars.kv_full(r.stage);
        if (lane == 0) mbar_arrive_expect_tx(bar, kLoadTile);
        __syncwarp();
        if (mine)
          tma_load_3d(dst_off + r.stage * kLoadTile, reinterpret_cast<const CUtensorMap*>(v ? map_v : map_k),
                      half * 64, static_cast<int32_t>((pos0 + static_cast<uint32_t>(tile) * kKeys) & in_page),
                      zz, bar);
        if (k8) {
          const int64_t er = older ? erow_v : erow;
          if (lane < kKeys / 8)
            cp_async8(base + L::kRawExp + r.stage * kKeys + lane * 8,
                      er >= 0 ? static_cast<const void*>((v ? c.ve : c.ke) + er) : a.q, er >= 0);
          cp_arrive(bar);
        }
        const uint32_t bit = 1u << r.stage;
        issued |= bit;
        if (by_hand) {
          hand |= bit;
          last = (last & ~bit) | (raw_phase & bit);
          raw_phase ^= bit;
        } else {
          hand &= ~bit;
          last = (last & ~bit) | (r.phase << r.stage);
        }
        r.step<L::kLoadStages>();
        return true;
      });
    }
    // What is on its way lands before the CTA goes, also after a timeout.
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (*ab.flag) {
      for (int s = 0; s < L::kLoadStages; ++s)
        if ((issued >> s) & 1u)
          wait_drain((hand >> s) & 1u ? bars.raw_full(s) : bars.kv_full(s), (last >> s) & 1u);
    }
  } else if (warp >= 8) {
    // ================= MMA issuer, query loader (and an idle warp) =================
    set_registers<Ro::kRegs, Ro::kRegsMain>();
    if (kShared && warp == kQueryWarp) {
      // Rows of several sequences, four to a lane and load; what is left of a tile
      // repeats the last one: rows that nobody reads.
      if constexpr (kShared) {
        const uint32_t bar = k8 ? bars.q_raw() : bars.q_full();
        Walk w;
        w.start_found(c, p.div, sh, run);
        uint32_t ord = 0;
        for (; !w.done(); ++ord, w.next(c, p.div)) {
          const Stretch s = c.list[w.b];
          const int tiles = kTwo && s.rows > 128 ? 2 : 1;
          int32_t y[2][4];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int at = MemberRow::row(a, s, min(x / 4 * 128 + lane * 4 + x % 4, s.rows - 1));
            y[x / 4][x % 4] = (at / a.rows1 * c.heads + w.unit) * a.rows1 + at % a.rows1;
          }
          if (!wait_warp(bars.q_empty(), (ord & 1u) ^ 1u, ab)) break;
          if (lane == 0) mbar_arrive_expect_tx(bar, tiles * L::kQTile);
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 2 * (D / 64); ++x)
            if (x / (D / 64) < tiles)
              tma_gather4(base + L::kQ0 + x * L::kQBox + lane * 512, &tq, x % (D / 64) * 64, y[x / (D / 64)], bar);
        }
        if (ord > 0) wait_drain(bar, (ord - 1u) & 1u);  // lands before the CTA goes, in any case
      }
    } else if (warp == kQueryWarp) {
      // Rows behind the head's belong to other heads or are zeros: rows of the
      // product that nobody reads.
      const uint32_t bar = k8 ? bars.q_raw() : bars.q_full();
      Walk w;
      w.start_found(c, p.div, sh, run);
      uint32_t ord = 0;
      for (; !w.done(); ++ord, w.next(c, p.div)) {
        if (!wait_warp(bars.q_empty(), (ord & 1u) ^ 1u, ab)) break;
        if (lane == 0) {
          const Unit un(a, p, w, rows);
          const bool two = kTwo && un.r0 + 128 < rows;
          mbar_arrive_expect_tx(bar, (two ? 2 : 1) * L::kQTile);
#pragma unroll 1
          for (int x = 0; x < (two ? 2 : 1) * (D / 64); ++x)
            tma_load_2d(base + L::kQ0 + x * L::kQBox, &tq, x % (D / 64) * 64,
                        static_cast<int32_t>(un.q0) + x / (D / 64) * 128, bar);
        }
        __syncwarp();
      }
      if (ord > 0) wait_drain(bar, (ord - 1u) & 1u);  // lands before the CTA goes, in any case
    } else if (warp == kMmaWarp) {
      // The whole warp walks along; one lane issues.
      const bool leader = elect_one();
      auto commit = [&](uint32_t bar) {
        if (leader) mma_commit(bar);
      };
      const uint64_t dQ0 = desc_sw128(base + L::kQ0, 16, 1024);
      const uint64_t dQ1 = desc_sw128(base + L::kQ1, 16, 1024);
      const uint64_t dK = desc_sw128(base + L::kKV, 16, 1024);
      const uint64_t dV = desc_sw128(base + L::kKV, L::kBox, 1024);
      const uint32_t tS0 = tmem, tS1 = tmem + 128, tO0 = tmem + 256, tO1 = tmem + 256 + D;
      Ring r;
      uint32_t unit = 0, np0 = 0, np1 = 0;  // units; P tiles taken per stream
      bool ok = true, any = false;
      Walk u;
      // wait for the next stage of the ring: its index, or -1
      auto take = [&]() {
        if (!wait_warp(bars.kv_full(r.stage), r.phase, ab)) return -1;
        const int s = r.stage;
        r.step<kS>();
        tc_fence_after();
        return s;
      };
      for (u.start_found(c, p.div, sh, run); ok && !u.done(); u.next(c, p.div), ++unit) {
        const int n = static_cast<int>(u.last - u.first);
        ok = wait_warp(bars.q_full(), unit & 1u, ab);
        if (!ok) break;
        any = true;
        int sk = take();
        if (sk < 0) {
          ok = false;
          break;
        }
        if (kTwo) {
          const bool two = second_tile(a, p, u, rows);
          uint64_t dk = dK + desc_step(sk * L::kTile);
          issue_qk<D, kKeys>(leader, tS0, dQ0, dk);
          commit(bars.s_full(0));
          if (two) {
            issue_qk<D, kKeys>(leader, tS1, dQ1, dk);
            commit(bars.s_full(1));
          }
          commit(bars.kv_empty(sk));
          if (n == 1) commit(bars.q_empty());
          for (int it = 0; it < n; ++it) {
            const int sv = take();
            if (sv < 0 || !wait_warp(bars.p_full(0), np0++ & 1u, ab)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t dv = dV + desc_step(sv * L::kTile);
            issue_pv<D, kKeys>(leader, tO0, tS0, dv, it > 0);
            const bool more = it + 1 < n;
            if (more) {
              sk = take();
              if (sk < 0) {
                ok = false;
                break;
              }
              dk = dK + desc_step(sk * L::kTile);
              issue_qk<D, kKeys>(leader, tS0, dQ0, dk);
              commit(bars.s_full(0));
            }
            if (two) {
              if (!wait_warp(bars.p_full(1), np1++ & 1u, ab)) {
                ok = false;
                break;
              }
              tc_fence_after();
              issue_pv<D, kKeys>(leader, tO1, tS1, dv, it > 0);
            }
            commit(bars.kv_empty(sv));
            if (more) {
              if (two) {
                issue_qk<D, kKeys>(leader, tS1, dQ1, dk);
                commit(bars.s_full(1));
              }
              commit(bars.kv_empty(sk));
              if (it + 2 == n) commit(bars.q_empty());  // the last scores
            }
          }
          if (ok) {
            commit(bars.o_full(0));
            if (two) commit(bars.o_full(1));
          }
        } else {
          issue_qk<D, kKeys>(leader, tS0, dQ0, dK + desc_step(sk * L::kTile));
          commit(bars.s_full(0));
          commit(bars.kv_empty(sk));
          if (n > 1) {
            sk = take();
            if (sk < 0) {
              ok = false;
              break;
            }
            issue_qk<D, kKeys>(leader, tS1, dQ0, dK + desc_step(sk * L::kTile));
            commit(bars.s_full(1));
            commit(bars.kv_empty(sk));
          }
          if (n <= 2) commit(bars.q_empty());
          for (int it = 0; it < n; ++it) {
            const int t = it & 1;
            const int sv = take();
            if (sv < 0 || !wait_warp(bars.p_full(t), (t ? np1++ : np0++) & 1u, ab)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t tS = t ? tS1 : tS0;
            issue_pv<D, kKeys>(leader, t ? tO1 : tO0, tS, dV + desc_step(sv * L::kTile), it > 1);
            commit(bars.kv_empty(sv));
            if (it + 2 < n) {
              sk = take();
              if (sk < 0) {
                ok = false;
                break;
              }
              issue_qk<D, kKeys>(leader, tS, dQ0, dK + desc_step(sk * L::kTile));
              commit(bars.s_full(t));
              commit(bars.kv_empty(sk));
              if (it + 3 == n) commit(bars.q_empty());  // the last scores
            }
          }
          if (ok) {
            commit(bars.o_full(0));
            if (n > 1) commit(bars.o_full(1));
          }
        }
      }
      if (!ok && any) {
        commit(bars.drain());
        wait_drain(bars.drain(), 0);
      }
    }
  } else {
    // ================= softmax =================
    set_registers<Ro::kRegs, Ro::kRegsSoftmax>();
    const int t = warp / 4, wq = warp % 4;
    const int row = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(t * 128);
    const uint32_t tO = tmem + lane_off + 256u + static_cast<uint32_t>(t * D);
    const uint64_t scale2 = pack_f32x2(a.scale_log2, a.scale_log2);
    float* xo = reinterpret_cast<float*>(gbase + L::kQ1);  // [2][128][33]
    float* xml = xo + 2 * 128 * 33;                        // [2][128][2]
    uint32_t ns = 0, no = 0, unit = 0, xc = 0, kt = 0;     // phases; K tiles before the unit
    bool ok = true;
    Walk& u = reinterpret_cast<Walk*>(gbase + L::kWalks)[warp];
    if (lane == 0) u.start_found(c, p.div, sh, run);
    __syncwarp();
    while (ok && !u.done()) {
      const int n = static_cast<int>(u.last - u.first);
      // the first tile of this part that holds drafts or the end
      const int border = static_cast<int>(
          min(max(u.seq.len / kKeys - u.first, int64_t{0}), static_cast<int64_t>(n)));
      const bool active = kTwo ? t == 0 || second_tile(a, p, u, rows) : t == 0 || n > 1;
      // What a thread's row is.  The wide form, whose loop has no registers to
      // spare, works it out again where it is needed.
      auto row_facts = [&]() {
        RowFacts f;
        if constexpr (kShared) {
          const MemberRow r(a, c.list[u.b], u.unit, (kTwo ? t * 128 : 0) + row);
          f = RowFacts{r.t, r.b, r.q, SeqInfo{u.seq.len, r.cnt}, r.q >= 0};
        } else {
          const Unit un(a, p, u, rows);
          const int64_t lrow = un.r0 + (kTwo ? t * 128 : 0) + row;  // row within the key head
          f.exists = lrow < rows;
          f.tok = f.exists ? static_cast<int>(lrow % c.T) : c.T;
          f.b = u.b;
          f.q = 0;
          f.seq = u.seq;
        }
        return f;
      };
      RowFacts facts = row_facts();
      const bool live = facts.tok < facts.seq.cnt;
      const bool warp_live = __any_sync(0xffffffffu, live);
      float m_ref = -INFINITY, l = 0.f;
      if constexpr (kWide) {
        if (active) {
          const WideTiles w{bars.s_full(t), bars.p_full(t), tS, tO, n, border, static_cast<int>(kt), ns, warp_live};
          const float2 ml = wide_tiles<D>(a, u, w, ab, gbase + L::kLeftOut, (kTwo ? t * 128 : 0) + row, kKeys);
          m_ref = ml.x;
          l = ml.y;
          ns += static_cast<uint32_t>(n);
          ok = *ab.flag == 0u && wait_warp(bars.o_full(t), no++ & 1u, ab);
          if (!ok) break;
          tc_fence_after();
        }
      } else if (active) {
        bool o_valid = false;
        for (int it = kTwo ? 0 : t; it < n; it += kTwo ? 1 : 2) {
          if (!wait_warp(bars.s_full(t), ns++ & 1u, ab)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (warp_live) {
            const uint32_t left = *reinterpret_cast<volatile uint32_t*>(
                gbase + L::kLeftOut + ((kt + it) & 31u) * 4);
            const bool masked = it >= border || left != 0u;
            if (masked) {  // scores that are not seen become -inf in TMEM
#pragma unroll 1
              for (int w = 0; w < kN; ++w) {
                const uint32_t seen =
                    seen_word(a, facts.seq, facts.b, facts.tok, (u.first + it) * kKeys + 32 * w, left >> (4 * w));
                uint32_t s[32];
                __syncwarp();
                tmem_ld32(tS + 32 * w, s);
                tmem_ld_wait();
                reg_fence(s, 32);
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  if (!((seen >> x) & 1u)) s[x] = __float_as_uint(-INFINITY);
                tmem_st32(tS + 32 * w, s);
              }
              tmem_st_wait();
            }
            // Two passes over the row's scores: the maximum, then the
            // probabilities, whose bf16 pairs take the place of scores that
            // have been read.  Rolled loops, for the instruction cache.
            float mx = -INFINITY;
#pragma unroll 1
            for (int w = 0; w < kN; w += 2) {
              uint32_t s[64];
              tmem_ld32(tS + 32 * w, s);
              tmem_ld32(tS + 32 * w + 32, s + 32);
              tmem_ld_wait();
              reg_fence(s, 64);
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 8]));
#pragma unroll
              for (int j = 16; j < 64; j += 16)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  v[e] = fmax3(v[e], __uint_as_float(s[j + e]), __uint_as_float(s[j + 8 + e]));
              mx = fmax3(mx, fmax3(v[0], v[1], v[2]), fmax3(fmax3(v[3], v[4], v[5]), v[6], v[7]));
            }
            float m_new = mx * a.scale_log2;
            const bool need = m_new > m_ref + kRescaleLog2;
            if (kShared) m_new += kHeadroom;
            if (__any_sync(0xffffffffu, need)) {
              const float alpha = need ? ex2(m_ref - m_new) : 1.f;
              if (o_valid) {
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                  uint32_t r[32];
                  tmem_ld32(tO + x, r);
                  tmem_ld_wait();
                  reg_fence(r, 32);
#pragma unroll
                  for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                  tmem_st32(tO + x, r);
                }
                tmem_st_wait();
              }
              if (need) {
                l *= alpha;
                m_ref = m_new;
              }
            }
            // a row that has seen no key yet keeps m_ref = -inf: p = 0, not NaN
            const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
            const uint64_t neg2 = pack_f32x2(neg, neg);
            uint64_t acc[2] = {0ull, 0ull};
            // 32 scores are on their way from TMEM while 32 are worked on
            uint32_t s0[32], s1[32];
            tmem_ld32(tS, s0);
            tmem_ld_wait();
            reg_fence(s0, 32);
#pragma unroll 1
            for (int w = 0; w < kN; w += 2) {
              tmem_ld32(tS + 32 * w + 32, s1);
              exp_part(s0, scale2, neg2, acc, tS + 16 * w);
              tmem_ld_wait();
              reg_fence(s1, 32);
              if (w + 2 < kN) tmem_ld32(tS + 32 * w + 64, s0);
              exp_part(s1, scale2, neg2, acc, tS + 16 * w + 16);
              tmem_ld_wait();
              reg_fence(s0, 32);
            }
            float a0, a1, a2, a3;
            unpack_f32x2(acc[0], a0, a1);
            unpack_f32x2(acc[1], a2, a3);
            l += (a0 + a1) + (a2 + a3);
            tmem_st_wait();
          }
          tc_fence_before();
          mbar_arrive(bars.p_full(t));
          o_valid = true;
        }
        if (!ok) break;
        if (!wait_warp(bars.o_full(t), no++ & 1u, ab)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      kt += static_cast<uint32_t>(n);
      if (kWide) facts = row_facts();
      if (!live) {
        m_ref = -INFINITY;
        l = 0.f;
      }
      const bool poisoned = poison[unit & 31] == unit + 1u;

      // ---- one query tile: the streams exchange halves of their states, so
      // that each finishes half of the columns
      const bool exchange = !kTwo && n > 1;
      float f0 = 1.f, f1 = 0.f;  // weights of this stream's and the other's sums
      if (kTwo ? active : t == 0 || exchange) {
        const Unit un(a, p, u, rows);
        const bool whole = u.whole(), finish = whole && !kShared;
        const int slot = u.slot(blockIdx.x);
        const int local = (kTwo ? t * 128 : 0) + row;
        const int first = exchange ? t * (D / 2) : 0;
        const int count = exchange ? D / 64 : D / 32;
        float inv = 1.f;
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
          const int x = first + 32 * i;
          uint32_t r[32];
          if (exchange) {
            // the other's half of this stream, through this stream's buffer
            if (!wait_warp(bars.x_empty(t), (xc & 1u) ^ 1u, ab)) {
              ok = false;
              break;
            }
            if (i == 0) {
              xml[(t * 128 + row) * 2] = m_ref;
              xml[(t * 128 + row) * 2 + 1] = l;
            }
            tmem_ld32(tO + (D / 2 - first) + 32 * i, r);
            tmem_ld_wait();
            reg_fence(r, 32);
            float* to = xo + (t * 128 + row) * 33;
#pragma unroll
            for (int e = 0; e < 32; ++e) to[e] = __uint_as_float(r[e]);
            mbar_arrive(bars.x_full(t));
          }
          tmem_ld32(tO + x, r);
          tmem_ld_wait();
          reg_fence(r, 32);
          if (exchange) {
            if (!wait_warp(bars.x_full(1 - t), xc & 1u, ab)) {
              ok = false;
              break;
            }
            if (i == 0) {
              const float m1 = xml[((1 - t) * 128 + row) * 2], l1 = xml[((1 - t) * 128 + row) * 2 + 1];
              const float ms = fmaxf(m_ref, m1);
              f0 = l == 0.f ? 0.f : ex2(m_ref - ms);
              f1 = l1 == 0.f ? 0.f : ex2(m1 - ms);
              l = f0 * l + f1 * l1;
              m_ref = ms;
            }
            const float* from = xo + ((1 - t) * 128 + row) * 33;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              r[e] = __float_as_uint(fmaf(f1, from[e], f0 * __uint_as_float(r[e])));
            }
            mbar_arrive(bars.x_empty(1 - t));
            ++xc;
          }
          if (i == 0 && finish) inv = l == 0.f ? 0.f : 1.f / l;
          // A row without a query may hold anything.  Of one that sees no key, or
          // a stream that it sees none of, the sums are 0; a weight of 0
          // multiplies all the same, since sums may be NaN.
          if (!live) {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0u;
          }
          if (k8) {  // back to the order of the head's elements
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const uint32_t y = r[e + 1];
              r[e + 1] = r[e + 2];
              r[e + 2] = y;
            }
          }
          if (poisoned && live) {
            // elements of drafts that were left out because they are not finite
            const uint32_t bad = poisoned_columns<k8, D>(a, u, facts.b, un.head, facts.tok, x, kKeys);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((bad >> e) & 1u) r[e] = 0x7fffffffu;
          }
          if (finish) {
            uint4 y[4];  // 8 columns each
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = make_uint4(
                  pack_bf16x2(__uint_as_float(r[8 * e + 0]) * inv, __uint_as_float(r[8 * e + 1]) * inv),
                  pack_bf16x2(__uint_as_float(r[8 * e + 2]) * inv, __uint_as_float(r[8 * e + 3]) * inv),
                  pack_bf16x2(__uint_as_float(r[8 * e + 4]) * inv, __uint_as_float(r[8 * e + 5]) * inv),
                  pack_bf16x2(__uint_as_float(r[8 * e + 6]) * inv, __uint_as_float(r[8 * e + 7]) * inv));
            // lane 4 i + j: the columns 8 j .. of rows 4 i .. 4 i + 3
            transpose4(y, lane);
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                                  (un.q0 + local - lane % 4) * D + x + 8 * (lane % 4));
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (un.r0 + local - lane % 4 + e < rows) dst[e * (D / 8)] = y[e];
            if (x == 0 && facts.exists)
              a.lse[un.q0 + local] = l == 0.f ? -INFINITY : (m_ref + __log2f(l)) * kLn2F;
          } else if (facts.exists) {
            float4* dst = reinterpret_cast<float4*>(slot_o(a, p, slot)) + x / 4 * p.rows + local;
            int64_t pitch = p.rows;
            if constexpr (kShared) {
              if (whole) {
                pitch = a.all_rows;
                dst = reinterpret_cast<float4*>(a.whole_o[c.list[u.b].first < 0]) + x / 4 * pitch + facts.q;
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e * pitch] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                            __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
            if (x == 0) {
              float* ml = slot_ml(a, p, slot) + 2 * local;
              if constexpr (kShared)
                if (whole) ml = a.whole_ml[c.list[u.b].first < 0] + 2 * facts.q;
              *reinterpret_cast<float2*>(ml) = make_float2(m_ref, l);
            }
          }
        }
        tc_fence_before();
      }
      ++unit;
      __syncwarp();
      if (lane == 0) u.next(c, p.div);
      __syncwarp();
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool k8, int D, bool kTwo, typename A>
cudaError_t launch_t(const A& a, const AttnPlan& plan, cudaStream_t s) {
  using L = Layout<k8, D, kTwo>;
  constexpr int kThreads = Roles<Form<k8, kTwo, A>::kWide>::kThreads;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(cache_tree_kernel<k8, D, kTwo, A>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  CUtensorMap tk, tv, tq;
  const int rows = (1 << a.c.page_shift) < L::kKeys ? 1 << a.c.page_shift : L::kKeys;
  if (!encode_pages(&tk, a.c.pages > 0 ? a.c.k : a.q, a.c, rows, k8) ||
      !encode_pages(&tv, a.c.pages > 0 ? a.c.v : a.q, a.c, rows, k8))
    return cudaErrorUnknown;
  AttnPlan p = plan;
  p.div.tile = L::kKeys;
  if constexpr (IsShared<A>::value) {
    if (!encode_single_rows(&tq, a.q, static_cast<int64_t>(a.c.B) * a.Hq * a.c.T, D)) return cudaErrorUnknown;
    cache_tree_kernel<k8, D, kTwo, A><<<p.div.ctas, kThreads, L::kSmem, s>>>(a, p, tk, tv, tq);
    return cudaGetLastError();
  } else {
    if (!encode_rows(&tq, a.q, static_cast<int64_t>(a.c.B) * a.Hq * a.c.T, D)) return cudaErrorUnknown;
    cache_tree_kernel<k8, D, kTwo, A><<<p.div.ctas, kThreads, L::kSmem, s>>>(a, p, tk, tv, tq);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_cache_tree_join(a, p, s) : e;
  }
}

template <bool k8, int D, typename A>
cudaError_t by_rows(const A& a, const AttnPlan& p, cudaStream_t s) {
  return p.rows == 256 ? launch_t<k8, D, true, A>(a, p, s) : launch_t<k8, D, false, A>(a, p, s);
}

template <typename A>
cudaError_t by_type(const A& a, const AttnPlan& p, bool k8, cudaStream_t s) {
  if (a.c.d == 128) return k8 ? by_rows<true, 128>(a, p, s) : by_rows<false, 128>(a, p, s);
  return k8 ? by_rows<true, 64>(a, p, s) : by_rows<false, 64>(a, p, s);
}

}  // namespace

cudaError_t launch_cache_tree(const CacheAttnArgs& a, bool k8, cudaStream_t s) {
  AttnPlan p;
  const int64_t rows = head_rows(a);
  p.rows = rows > 128 ? 256 : 128;
  p.row_tiles = static_cast<int>((rows + p.rows - 1) / p.rows);
  p.div.units = a.c.heads * p.row_tiles;
  p.div.ctas = kTreeCtas;
  return by_type(a, p, k8, s);
}

SharedShape tree_shape(int d, bool two) {
  const int tile = two || d == 64 ? 128 : 64;
  return SharedShape{tile, two ? 256 : 128, kTreeCtas, 768 / tile, true};
}

cudaError_t launch_shared_tree(const SharedAttnArgs& a, const AttnPlan& p, bool k8, cudaStream_t s) {
  return by_type(a, p, k8, s);
}

}  // namespace ra
