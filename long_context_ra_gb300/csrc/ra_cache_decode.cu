// Attention over the paged cache for few query rows per key head (a decode
// step of grouped-query heads, a handful of drafts): bf16 queries, bf16 or
// 8-bit cache.
//
// Bound by the bytes of the cache: with 16 rows a byte of K or V feeds 16 to
// 32 multiply-adds.  So the kernel is built around the loads.  A CTA is 4
// warps, each on keys of its own (32 of every tile of 128) with a state of its
// own, joined at the end of a unit: nothing but the loads is waited for in
// between.  Each warp brings its chunks of 32 keys, K and V in turn, with
// cp.async through a ring of kStages places in shared memory; the page numbers
// of the next chunks are held by the 32 lanes, one coalesced load ahead.  32
// keys make four score products and two value products independent of one
// another, which two warps per scheduler need to hide the latency of each.
//
// The products are m16n8k16 mma with the 16 query rows as M, which leaves
// the order of the contracted index free: a lane takes 16 contiguous bytes of
// a key row as its part of several k-steps (K), and 16 contiguous bytes of
// four key rows as its column of several n-tiles (V), so every shared-memory
// read is 16 bytes wide and needs no transposing load.  The pieces of a row
// are placed by XOR so that these reads meet no bank twice.
//
// 8-bit rows become f16 in registers (every e4m3 value is an f16); the row
// scales are powers of two and act on the scores (K) and on the exponents of
// the probabilities (V).  Queries are scaled per row to at most 2^15, so that
// bf16's 8 bits fit f16 down to 2^-29 of the row's maximum.  The f16
// probabilities carry the V scale: they are kept relative to their own
// running maximum (of s + e_v) at 2^7, so a weight is rounded to 11 bits down
// to 2^-21 of the largest one and lost below 2^-32 of it.  bf16
// probabilities are rounded to 8 bits; sums are fp32 of unrounded values.
//
// As in the forward, the reference of the exponentials moves only when a
// score passes it by more than 2^8: a vote per chunk instead of a row maximum.
//
// Measured, 32 ragged sequences of up to 32768, 8 key heads of 128, 4 queries
// each: 8-bit cache (1.25 GB) 220 us, 5.7 TB/s, 84 % of the copy rate.  With 64
// keys a chunk it took 348 us, with 32 and V behind all of K 303; the packed
// conversions made that 230, leaving out the second 8 rows where a unit has none
// 220.  A unit costs some 6 us beside its tiles, of which the look-up of its first
// pages goes on while the one ahead is joined (96 sequences of up to 2048, 8 key
// heads, 8 bits: 179 -> 165 us with both).  Pages of 32 rows and more are alike; smaller ones
// take a look-up per 16-byte piece (32 sequences of 16384, 8 bits: 188 us with
// pages of 32 to 256, 320 of 8 or 16; bf16 313 and 453).  One sequence of 1000 takes 12 us, most of it the
// two launches and the chain of look-up, load and join.

#include "ra_cache_attn.cuh"
#include "sm103_ptx.cuh"

namespace ra {
namespace {

using namespace ptx;

constexpr int kRows = 16;
constexpr int kWarps = 4;
constexpr int kChunk = 32;
constexpr int kTile = kWarps * kChunk;
constexpr int kThreads = kWarps * 32;
constexpr float kSlack = 8.f;      // log2: how far a score may pass the reference
constexpr float kF16Offset = 7.f;  // log2: f16 weights are at most 2^(kSlack + kF16Offset)

template <bool k8, int D>
struct Shape {
  static constexpr int kRowBytes = k8 ? D : 2 * D;
  static constexpr int kPieces = kRowBytes / 16;
  static constexpr int kSide = kChunk * kRowBytes;          // K or V of a chunk
  static constexpr int kStage = kSide + (k8 ? kChunk : 0);  // + its exponent bytes
  static constexpr int kStages = kSide > 4096 ? 3 : 6;      // two CTAs fit an SM
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kLd = D + 4;                          // row pitch of the joined states
  static constexpr int kJoin = kWarps * kRows * (kLd + 2) * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
  static constexpr int kTilesN = D / 8;
  // Byte offset of 16-byte piece c of row r.  K is read as (two neighbouring
  // rows, four pieces), V as (four rows 2 apart, two pieces) per phase.
  __device__ static int at_k(int r, int c) {
    if (kPieces == 4) return (r >> 1) * 128 + ((((r & 1) << 2) + c) ^ (((r >> 1) & 3) << 1)) * 16;
    return r * kRowBytes + (c ^ ((r & 1) << 2)) * 16;
  }
  __device__ static int at_v(int r, int c) {
    if (kPieces == 4) return at_k(r, c);
    return r * kRowBytes + (c ^ (r & 6)) * 16;
  }
  // Element of the head that column c (0 .. 7) of n-tile nn stands for.
  __device__ static int column(int nn, int c) {
    if (k8) return c * (D / 8) + nn;
    return (nn / 8) * 64 + c * 8 + nn % 8;
  }
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 x;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at));
  return x;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at));
  return x;
}

// c += a b, 16 x 8 x 16, fp32 sums.
template <bool k8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (k8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <bool k8>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  return k8 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// Halves of x that are not finite, as 0xffff masks.
template <bool k8>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  constexpr uint32_t e = k8 ? 0x7c00u : 0x7f80u;
  return ((x & e) == e ? 0xffffu : 0u) | (((x >> 16) & e) == e ? 0xffff0000u : 0u);
}

// B fragments of the n-tiles from the value rows of four keys, in order.
// kWords 32-bit words of each row; f(nn, b0, b1) is called for each n-tile.
template <bool k8, int kWords, typename F>
__device__ __forceinline__ void each_value_tile(const uint32_t (&w)[4][kWords], F f) {
#pragma unroll
  for (int q = 0; q < kWords; ++q) {
    if (k8) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t sel = z ? 0x7362u : 0x5140u;  // bytes (key 0, key 1) of two elements
        const uint32_t x = __byte_perm(w[0][q], w[1][q], sel);
        const uint32_t y = __byte_perm(w[2][q], w[3][q], sel);
        uint32_t x0, x1, y0, y1;
        e4m3x4_to_f16x4(x, x0, x1);
        e4m3x4_to_f16x4(y, y0, y1);
        f(4 * q + 2 * z, x0, y0);
        f(4 * q + 2 * z + 1, x1, y1);
      }
    } else {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t sel = z ? 0x7632u : 0x5410u;  // halves (key 0, key 1) of one element
        f(2 * q + z, __byte_perm(w[0][q], w[1][q], sel), __byte_perm(w[2][q], w[3][q], sel));
      }
    }
  }
}

template <bool k8, int D, typename A>
__global__ void __launch_bounds__(kThreads, 2)
    cache_decode_kernel(const __grid_constant__ A a,
                        const __grid_constant__ AttnPlan p) {
  using S = Shape<k8, D>;
  // whole lines: a base that is only 16-byte aligned costs 5 % (238 us, not 227)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ DivisionShared sh;
  constexpr bool kShared = IsShared<A>::value;
  const auto& c = paged(a);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const uint32_t ring = smem_u32(smem) + warp * (S::kStages * S::kStage);
  const int64_t rows = head_rows(a);

  allow_join();
  const int64_t run = division_start(c, p.div, blockIdx.x, sh);
  typename IsShared<A>::Walk u;
  u.start(c, p.div, sh, run);

  // ---- page numbers.  A chunk lies in `per` pages (granules of min(page,
  // 32) rows); lane i holds granule base * per + i.  A unit's first are looked up
  // before the one ahead of it is joined.
  const int gshift = min(c.page_shift, 5), per = kChunk >> gshift;
  auto look_up = [&](const typename IsShared<A>::Walk& w, int base) {
    const int chunk = base + lane / per;
    const int64_t at = (w.first + chunk) * kTile + warp * kChunk + ((lane % per) << gshift);
    if (w.first + chunk >= w.last || at >= w.seq.keys()) return -1;
    const int64_t col = at >> c.page_shift;
    const int page = col < columns_of(c, w.b) ? pages_of(c, w.b)[col] : -1;
    if (page >= 0 && page < c.pages) return page;
    flag_page(c.status);
    return -1;
  };
  const int batch = 32 / per;  // chunks whose pages the lanes hold
  int pg = -1, nx = -1;
  if (!u.done()) {
    pg = look_up(u, 0);
    nx = look_up(u, batch);
  }
  while (!u.done()) {
    const int head = u.unit / p.row_tiles;
    const int64_t r0 = static_cast<int64_t>(u.unit % p.row_tiles) * kRows;
    const int64_t q0 = (static_cast<int64_t>(u.b) * c.heads + head) * rows + r0;
    const int64_t keys = u.seq.keys();
    const int n = static_cast<int>(u.last - u.first);  // chunks of this warp
    const int64_t key0 = u.first * kTile + warp * kChunk;

    uint32_t left_out = 0;       // of the chunk loaded last: a bit per 8 rows not in the cache
    uint32_t left_ring = 0;      // the same of the chunks under way, 4 bits each, newest lowest
    const int64_t in_page = (int64_t{1} << c.page_shift) - 1;
    auto issue = [&](int m) {  // item m: K (even) or V (odd) of chunk m / 2
      const int i = m >> 1;
      const bool v = m & 1;
      if (!v && i > 0 && i % batch == 0) {
        pg = nx;
        nx = look_up(u, i + batch);
      }
      const int64_t pos = key0 + static_cast<int64_t>(i) * kTile;
      const uint32_t dst = ring + (m % S::kStages) * S::kStage;
      const uint8_t* src = static_cast<const uint8_t*>(v ? c.v : c.k);
      const uint8_t* exps = v ? c.ve : c.ke;
      const int first = (i % batch) * per;
      const int page0 = __shfl_sync(0xffffffffu, pg, first);
      if (per == 1 && page0 >= 0 && pos + kChunk <= keys) {
        // the chunk is 32 rows of one page
        const int64_t row = ((static_cast<int64_t>(page0) * c.heads + head) << c.page_shift) + (pos & in_page);
        const uint8_t* p0 = src + row * S::kRowBytes + lane * 16;
#pragma unroll
        for (int x = 0; x < S::kSide / 512; ++x) {
          const int piece = x * 32 + lane, r = piece / S::kPieces, pc = piece % S::kPieces;
          cp_async16(dst + (v ? S::at_v(r, pc) : S::at_k(r, pc)), p0 + x * 512, true);
        }
        if (k8 && lane < 4) cp_async8(dst + S::kSide + lane * 8, exps + row + lane * 8, true);
        if (!v) left_out = 0;
      } else {
        uint32_t out = 0;
#pragma unroll 1
        for (int x = 0; x < S::kSide / 512; ++x) {
          const int piece = x * 32 + lane, r = piece / S::kPieces, pc = piece % S::kPieces;
          const int page = __shfl_sync(0xffffffffu, pg, first + (r >> gshift));
          const bool real = pos + r < keys && page >= 0;
          const int64_t row =
              ((static_cast<int64_t>(page) * c.heads + head) << c.page_shift) + ((pos + r) & in_page);
          cp_async16(dst + (v ? S::at_v(r, pc) : S::at_k(r, pc)),
                     real ? src + row * S::kRowBytes + pc * 16 : a.q, real);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // rows 8 x .. 8 x + 7
          const int page = __shfl_sync(0xffffffffu, pg, first + ((8 * x) >> gshift));
          const bool real = pos + 8 * x < keys && page >= 0;
          if (page < 0) out |= 1u << x;
          const int64_t row =
              ((static_cast<int64_t>(page) * c.heads + head) << c.page_shift) + ((pos + 8 * x) & in_page);
          if (k8 && lane == x)
            cp_async8(dst + S::kSide + x * 8, real ? static_cast<const void*>(exps + row) : a.q, real);
        }
        if (!v) left_out = out;
      }
      if (!v) left_ring = (left_ring << 4) | left_out;
    };

#pragma unroll 1
    for (int m = 0; m < S::kStages - 1; ++m) {
      if (m < 2 * n) issue(m);
      cp_commit();
    }
    // waits for item m and brings the item kStages - 1 behind it
    auto arrive = [&](int m) {
      cp_wait<S::kStages - 2>();
      __syncwarp();
      if (m + S::kStages - 1 < 2 * n) issue(m + S::kStages - 1);
      cp_commit();
      return ring + (m % S::kStages) * S::kStage;
    };

    // ---- queries as A fragments, in the order in which K rows are read
    uint32_t qf[D / 16][4];
    float scale[2];
    int tq[2], mask_b[2];  // a row's token and sequence
    SeqInfo seq[2];        // the context and new tokens that it may see
    bool two;              // rows 8 .. 15 hold queries too
    if constexpr (kShared)
      two = c.list[u.b].rows > 8;
    else
      two = rows - r0 > 8;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) qf[st][1] = qf[st][3] = 0u;
    scale[1] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !two) break;
      bool real;
      int64_t at;
      if constexpr (kShared) {
        const MemberRow r(a, c.list[u.b], u.unit, g + 8 * h);
        real = r.q >= 0;
        at = r.q;
        tq[h] = r.t;
        mask_b[h] = r.b;
        seq[h] = SeqInfo{u.seq.len, r.cnt};
      } else {
        const int64_t row = r0 + g + 8 * h;
        real = row < rows;
        at = q0 + g + 8 * h;
        tq[h] = real ? static_cast<int>(row % c.T) : c.T;
        mask_b[h] = u.b;
        seq[h] = u.seq;
      }
      const uint8_t* src = static_cast<const uint8_t*>(a.q) + at * D * 2;
      uint32_t amax = 0;
#pragma unroll
      for (int st = 0; st < D / 16; ++st) {
        const int d0 = k8 ? 64 * (st / 4) + 16 * t + 4 * (st % 4) : 32 * (st / 2) + 8 * t + 4 * (st % 2);
        const uint2 x = real ? *reinterpret_cast<const uint2*>(src + 2 * d0) : make_uint2(0u, 0u);
        qf[st][h] = x.x;
        qf[st][2 + h] = x.y;
        if (k8) {
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const uint32_t m = ((z & 2 ? x.y : x.x) >> (16 * (z & 1))) & 0x7fffu;
            if (m < 0x7f80u && m > amax) amax = m;
          }
        }
      }
      scale[h] = a.scale_log2;
      if (k8) {
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // the largest finite element goes to [2^14, 2^15)
        const int e = amax ? min(max(268 - static_cast<int>(amax >> 7), 1), 253) : 127;
        const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
        scale[h] *= __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
        for (int st = 0; st < D / 16; ++st)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t x = qf[st][2 * z + h];
            qf[st][2 * z + h] = pack_f16x2(__uint_as_float(x << 16) * up,
                                           __uint_as_float(x & 0xffff0000u) * up);
          }
      }
    }

    float m[2] = {-INFINITY, -INFINITY};   // reference of l (log2)
    float mo[2] = {-INFINITY, -INFINITY};  // reference of o (k8; else it is m)
    float l[2] = {0.f, 0.f};               // this lane's share
    float o[S::kTilesN][4];
#pragma unroll
    for (int nn = 0; nn < S::kTilesN; ++nn)
#pragma unroll
      for (int z = 0; z < 4; ++z) o[nn][z] = 0.f;

#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const uint32_t kb = arrive(2 * i);
      const int64_t pos = key0 + static_cast<int64_t>(i) * kTile;
      // chunks loaded but not worked on yet, this one the oldest: its bits
      const int newest = min((2 * i + S::kStages - 1) >> 1, n - 1);
      const uint32_t out = (left_ring >> (4 * (newest - i))) & 15u;

      // ---- scores of 32 keys (four n-tiles)
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int z = 0; z < 4; ++z) s[j][z] = 0.f;
#pragma unroll
      for (int x = 0; x < S::kPieces / 4; ++x) {
        uint4 w4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w4[j] = lds128(kb + S::at_k(8 * j + g, t + 4 * x));
#pragma unroll
        for (int z = 0; z < (k8 ? 4 : 2); ++z) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w[4] = {w4[j].x, w4[j].y, w4[j].z, w4[j].w};
            if (k8) {
              uint32_t b0, b1;
              e4m3x4_to_f16x4(w[z], b0, b1);
              mma16816<k8>(s[j], qf[4 * x + z], b0, b1);
            } else {
              mma16816<k8>(s[j], qf[2 * x + z], w[2 * z], w[2 * z + 1]);
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float ks[2] = {1.f, 1.f};
        if (k8) {
          const uint32_t ek = lds16(kb + S::kSide + 8 * j + 2 * t);
          ks[0] = exp_scale(ek & 255u);
          ks[1] = exp_scale(ek >> 8);
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) s[j][z] *= k8 ? scale[0] * ks[z] : scale[0];
        if (two) {
#pragma unroll
          for (int z = 0; z < 2; ++z) s[j][2 + z] *= k8 ? scale[1] * ks[z] : scale[1];
        }
      }
      const uint32_t vb = arrive(2 * i + 1);
      float ev[4][2];  // log2 of the V scales of this lane's columns
      if (k8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t e2 = lds16(vb + S::kSide + 8 * j + 2 * t);
          ev[j][0] = static_cast<float>(static_cast<int>(e2 & 255u) - 127);
          ev[j][1] = static_cast<float>(static_cast<int>(e2 >> 8) - 127);
        }
      }
      // every row sees every key, but for drafts, the end, and pages left out
      const bool all_seen = pos + kChunk <= u.seq.len && out == 0;
      uint32_t seen = 0xffffu;  // bit 4 j + z: of score s[j][z]
      if (!all_seen) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int j = x / 4, z = x % 4;
          if (z >= 2 && !two) continue;
          if (((out >> j) & 1u) || !sees(a, seq[z / 2], mask_b[z / 2], tq[z / 2], pos + 8 * j + 2 * t + z % 2)) {
            seen &= ~(1u << x);
            s[j][z] = -INFINITY;
          }
        }
      }

      // ---- reference, probabilities, sums
      bool pass = false;
      float xm[2], ym[2];  // this lane's largest s, and s + ev
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        xm[h] = -INFINITY;
        ym[h] = -INFINITY;
        if (h == 1 && !two) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xm[h] = fmax3(xm[h], s[j][2 * h], s[j][2 * h + 1]);
          if (k8) ym[h] = fmax3(ym[h], s[j][2 * h] + ev[j][0], s[j][2 * h + 1] + ev[j][1]);
        }
        pass = pass || xm[h] > m[h] + kSlack;
        if (k8) pass = pass || ym[h] > mo[h] + kSlack;
      }
      if (__any_sync(0xffffffffu, pass)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) break;
          float x = fmaxf(m[h], xm[h]), y = fmaxf(mo[h], ym[h]);
#pragma unroll
          for (int w = 1; w < 4; w <<= 1) {
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
            if (k8) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, w));
          }
          const float al = m[h] == x ? 1.f : exp2f(m[h] - x);
          const float ao = k8 ? (mo[h] == y ? 1.f : exp2f(mo[h] - y)) : al;
          l[h] *= al;
          m[h] = x;
          mo[h] = y;
#pragma unroll
          for (int nn = 0; nn < S::kTilesN; ++nn) {
            o[nn][2 * h] *= ao;
            o[nn][2 * h + 1] *= ao;
          }
        }
      }
      uint32_t pf[2][4];  // A fragments of the two halves of the chunk
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !two) {
          pf[0][1] = pf[0][3] = pf[1][1] = pf[1][3] = 0u;
          break;
        }
        const float ref = m[h] == -INFINITY ? 0.f : m[h];
        const float refo = mo[h] == -INFINITY ? 0.f : mo[h] - kF16Offset;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p0 = ex2(s[j][2 * h] - ref), p1 = ex2(s[j][2 * h + 1] - ref);
          l[h] += p0 + p1;
          pf[j / 2][2 * (j % 2) + h] = k8 ? pack_p<k8>(ex2(s[j][2 * h] + ev[j][0] - refo),
                                                       ex2(s[j][2 * h + 1] + ev[j][1] - refo))
                                          : pack_p<k8>(p0, p1);
        }
      }

      // ---- values: this lane's columns of keys 2t, 2t + 1, 8 + 2t, 9 + 2t
      // of each half; kWords 32-bit words of a key row at a time
      constexpr int kWords = D == 64 && k8 ? 2 : 4;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int part = 0; part < S::kRowBytes / 32 / kWords; ++part) {
          uint32_t w[4][kWords];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int r = 16 * half + 8 * (z / 2) + 2 * t + (z & 1);
            if (kWords == 2) {
              const uint2 x = lds64(vb + S::at_v(r, g / 2) + 8 * (g & 1));
              w[z][0] = x.x;
              w[z][1] = x.y;
            } else {
              const uint4 y = lds128(vb + S::at_v(r, g + 8 * part));
              w[z][0] = y.x;
              w[z][1] = y.y;
              w[z][kWords - 2] = y.z;
              w[z][kWords - 1] = y.w;
            }
          }
          bool poison = false;
          if (!all_seen) {
            each_value_tile<k8, kWords>(w, [&](int, uint32_t b0, uint32_t b1) {
              poison = poison || not_finite<k8>(b0) || not_finite<k8>(b1);
            });
            poison = __any_sync(0xffffffffu, poison);
          }
          if (!poison) {
            each_value_tile<k8, kWords>(w, [&](int nn, uint32_t b0, uint32_t b1) {
              mma16816<k8>(o[8 * part + nn], pf[half], b0, b1);
            });
          } else {
            // Values that are not finite reach the rows that see their key and
            // no others: they are left out of the product, and a second product
            // counts, per row and column, those the row sees.
            constexpr uint32_t one = k8 ? 0x3c003c00u : 0x3f803f80u;
            uint32_t sf[4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t two = seen >> (4 * (2 * half + j) + 2 * h);
                sf[2 * j + h] = one & ((two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u));
              }
            each_value_tile<k8, kWords>(w, [&](int nn, uint32_t b0, uint32_t b1) {
              const uint32_t n0 = not_finite<k8>(b0), n1 = not_finite<k8>(b1);
              float cnt[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816<k8>(cnt, sf, one & n0, one & n1);
              mma16816<k8>(o[8 * part + nn], pf[half], b0 & ~n0, b1 & ~n1);
#pragma unroll
              for (int z = 0; z < 4; ++z)
                if (cnt[z] > 0.f) o[8 * part + nn][z] = NAN;
            });
          }
        }
      }
    }

    typename IsShared<A>::Walk following = u;
    following.next(c, p.div);
    if (!following.done()) {
      pg = look_up(following, 0);
      nx = look_up(following, batch);
    }

    // ---- join the four warps' states
    cp_wait<0>();
    __syncthreads();
    float* js = reinterpret_cast<float*>(smem);          // [warp][row][kLd] o relative to m
    float* jm = js + kWarps * kRows * S::kLd;             // [warp][row][2]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !two) break;
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      const bool dead = tq[h] >= seq[h].cnt;  // no query: an empty state
      if (dead) {
        m[h] = -INFINITY;
        l[h] = 0.f;
      }
      const int row = warp * kRows + g + 8 * h;
      if (t == 0) {
        jm[2 * row] = m[h];
        jm[2 * row + 1] = l[h];
      }
      const float f = k8 && mo[h] != -INFINITY ? exp2f(mo[h] - kF16Offset - m[h]) : 1.f;
#pragma unroll
      for (int nn = 0; nn < S::kTilesN; ++nn)
#pragma unroll
        for (int z = 0; z < 2; ++z)
          js[row * S::kLd + S::column(nn, 2 * t + z)] = dead ? 0.f : o[nn][2 * h + z] * f;
    }
    __syncthreads();
    {
      const int r = threadIdx.x / 8, x0 = (threadIdx.x % 8) * 4;
      bool here = r0 + r < rows;
      int64_t q_row = 0;  // its place in q (stretches)
      if constexpr (kShared) {
        q_row = MemberRow(a, c.list[u.b], u.unit, r).q;
        here = q_row >= 0;
      }
      if (here) {
        float ms = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) ms = fmaxf(ms, jm[2 * (w * kRows + r)]);
        const float ref = ms == -INFINITY ? 0.f : ms;
        float f[kWarps], ls = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float lw = jm[2 * (w * kRows + r) + 1];
          f[w] = lw == 0.f ? 0.f : exp2f(jm[2 * (w * kRows + r)] - ref);
          ls += f[w] * lw;
        }
        const bool whole = u.whole(), finish = whole && !kShared;
        const float fin = finish ? (ls == 0.f ? 0.f : 1.f / ls) : 1.f;
        const int slot = u.slot(blockIdx.x);
        if (threadIdx.x % 8 == 0) {
          if (finish) {
            a.lse[q0 + r] = ls == 0.f ? -INFINITY : (ms + log2f(ls)) * kLn2F;
          } else {
            float* ml = slot_ml(a, p, slot) + 2 * r;
            if constexpr (kShared)
              if (whole) ml = a.whole_ml[c.list[u.b].first < 0] + 2 * q_row;
            ml[0] = ms;
            ml[1] = ls;
          }
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(js + (w * kRows + r) * S::kLd + 32 * x + x0);
            // a weight of 0 too: y may be NaN, and is 0 without a seen key
            v[0] = fmaf(f[w], y.x, v[0]);
            v[1] = fmaf(f[w], y.y, v[1]);
            v[2] = fmaf(f[w], y.z, v[2]);
            v[3] = fmaf(f[w], y.w, v[3]);
          }
          if (finish) {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (q0 + r) * D + 32 * x + x0) =
                make_uint2(pack_bf16x2(v[0] * fin, v[1] * fin), pack_bf16x2(v[2] * fin, v[3] * fin));
          } else {
            float4* dst = reinterpret_cast<float4*>(slot_o(a, p, slot) + r * D + 32 * x + x0);
            if constexpr (kShared)
              if (whole) dst = reinterpret_cast<float4*>(a.whole_o[c.list[u.b].first < 0]) + (8 * x + x0 / 4) * a.all_rows + q_row;
            *dst = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
      }
    }
    __syncthreads();
    u = following;
  }
}

template <bool k8, int D, typename A>
cudaError_t launch_t(const A& a, const AttnPlan& p, cudaStream_t s) {
  using S = Shape<k8, D>;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(cache_decode_kernel<k8, D, A>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cache_decode_kernel<k8, D, A><<<p.div.ctas, kThreads, S::kSmem, s>>>(a, p);
  e = cudaGetLastError();
  if constexpr (IsShared<A>::value)
    return e;
  else
    return e == cudaSuccess ? launch_cache_attn_join(a, p, true, s) : e;
}

template <typename A>
cudaError_t by_type(const A& a, const AttnPlan& p, bool k8, cudaStream_t s) {
  if (a.c.d == 128) return k8 ? launch_t<true, 128>(a, p, s) : launch_t<false, 128>(a, p, s);
  return k8 ? launch_t<true, 64>(a, p, s) : launch_t<false, 64>(a, p, s);
}

}  // namespace

cudaError_t launch_cache_decode(const CacheAttnArgs& a, bool k8, cudaStream_t s) {
  AttnPlan p;
  p.rows = kRows;
  p.row_tiles = static_cast<int>((head_rows(a) + kRows - 1) / kRows);
  p.div.units = a.c.heads * p.row_tiles;
  p.div.tile = kTile;
  p.div.ctas = kDecodeCtas;
  return by_type(a, p, k8, s);
}

SharedShape decode_shape(bool k8) { return SharedShape{kTile, kRows, kDecodeCtas, k8 ? 6 : 8, false}; }

cudaError_t launch_shared_decode(const SharedAttnArgs& a, const AttnPlan& p, bool k8, cudaStream_t s) {
  return by_type(a, p, k8, s);
}

}  // namespace ra
