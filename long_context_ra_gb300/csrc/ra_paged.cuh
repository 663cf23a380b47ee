// Device helpers of the paged cache: a position's row, the 8-bit format, and
// the division of a ragged batch's key tiles among the CTAs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "ra_internal.h"
#include "ra_serve.h"

namespace ra {

// A timeout, whose results are invalid, is not replaced.
__device__ __forceinline__ void flag_page(int* status) { atomicCAS(status, 0, kStatusPage); }

// Row of head 0 of position `pos` of sequence b in the cache (add
// h << page_shift for head h), or -1, with the status word set, for a
// position or page outside the cache.
__device__ __forceinline__ int64_t cache_row(const PagedArgs& c, int b, int64_t pos) {
  const int64_t col = pos >> c.page_shift;
  if (col < c.width) {
    const int64_t page = c.table[static_cast<int64_t>(b) * c.width + col];
    if (page >= 0 && page < c.pages)
      return ((page * c.heads) << c.page_shift) + (pos & ((int64_t{1} << c.page_shift) - 1));
  }
  flag_page(c.status);
  return -1;
}

// Context and new tokens of sequence b; a sequence with lens < 0 has none.
struct SeqInfo {
  int64_t len;
  int cnt;
  __device__ int64_t keys() const { return len + cnt; }
};

__device__ __forceinline__ SeqInfo sequence(const PagedArgs& c, int b) {
  SeqInfo s;
  const int32_t len = c.lens[b];
  const int32_t cnt = c.count ? c.count[b] : c.T;
  s.len = len < 0 ? 0 : len;
  s.cnt = len < 0 ? 0 : max(0, min(cnt, c.T));
  return s;
}

// 2^(e - 127) of an exponent byte.
__device__ __forceinline__ float exp_scale(uint32_t e) {
  return __uint_as_float(e ? e << 23 : 0x00400000u);
}

// Exponent byte of a row with largest magnitude amax: the smallest e >= -126
// with amax <= 448 * 2^e (448 = 1.75 * 2^8, the largest e4m3 value).
__device__ __forceinline__ uint32_t row_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 1));
}

__device__ __forceinline__ uint32_t pack_e4m3x4(const float* x) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The four e4m3 bytes of w as two pairs of f16 (exact: every e4m3 value is an
// f16).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void unpack_e4m3x4(uint32_t w, float* x) {
  uint32_t h[2];
  e4m3x4_to_f16x4(w, h[0], h[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// 8 consecutive floats.
__device__ __forceinline__ void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// kV consecutive elements of a row as they lie in memory: loaded with wide
// loads that bypass L1, unpacked to floats when they are used, so that many
// can be on their way.
template <typename E, int kV>
struct Packed {
  static constexpr int kBytes = kV * static_cast<int>(sizeof(E));
  static constexpr int kWords = kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const void* p) {
    if (kBytes == 8) {
      asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
                   : "=r"(w[0]), "=r"(w[1])
                   : "l"(p));
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                     : "l"(static_cast<const uint8_t*>(p) + 4 * i));
    }
  }
  __device__ __forceinline__ void store(void* p) const {
    if (kBytes == 8) {
      *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p) + 4 * i) =
            make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
  __device__ __forceinline__ void get(float (&x)[kV]) const {
    if (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] = __uint_as_float(w[i % kWords]);
    } else if (sizeof(E) == 2) {
#pragma unroll
      for (int i = 0; i < kV; i += 2) {
        x[i] = __uint_as_float(w[(i / 2) % kWords] << 16);
        x[i + 1] = __uint_as_float(w[(i / 2) % kWords] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kV; i += 4) unpack_e4m3x4(w[(i / 4) % kWords], x + i);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[kV]) {
    if (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < kV; ++i) w[i % kWords] = __float_as_uint(x[i]);
    } else if (sizeof(E) == 2) {
#pragma unroll
      for (int i = 0; i < kV; i += 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[i], x[i + 1]);
        w[(i / 2) % kWords] = *reinterpret_cast<const uint32_t*>(&h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kV; i += 4) w[(i / 4) % kWords] = pack_e4m3x4(x + i);
    }
  }
};

// ------------------------------------------------------------ work division
//
// A unit is one tile of query rows of one key head of one sequence; it walks
// the sequence's key tiles.  The tiles of all units, in the order (sequence,
// unit, tile), are cut into equal runs, one per CTA, so that a batch of
// unlike lengths keeps every CTA busy for the same time.  A CTA meets at
// most one unit that began before its run (its state goes to slot 2c) and
// one that goes on behind it (slot 2c + 1); the units between are whole.
struct Division {
  int units;     // per sequence: key heads x row tiles
  int tile;      // keys per tile
  int ctas;
};

__device__ __forceinline__ int64_t tiles_of(const SeqInfo& s, const Division& v) {
  const int64_t n = s.keys();
  return n <= v.tile ? 1 : (n + v.tile - 1) / v.tile;  // an empty sequence has one empty tile
}
__device__ __forceinline__ int64_t seq_tiles(const PagedArgs& c, const Division& v, int b) {
  return tiles_of(sequence(c, b), v);
}

__device__ __forceinline__ int64_t run_length(const Division& v, int64_t total) {
  return (total + v.ctas - 1) / v.ctas;
}

// Shared scratch of the block-wide sums below.
struct DivisionShared {
  int64_t warp[32];
  int64_t total;  // tiles of all sequences (one unit each)
  int64_t off;    // of the CTA's first tile within its sequence's tiles
  int b;          // sequence of the CTA's first tile
  SeqInfo seq;
  int64_t run;    // tiles of a CTA
};

// Inclusive scan of one value per thread; sh.total = the sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, DivisionShared& sh) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = (blockDim.x + 31) / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh.warp[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int i = 0; i < warps; ++i) {
    if (i < warp) before += sh.warp[i];
    all += sh.warp[i];
  }
  if (threadIdx.x == 0) sh.total = all;
  return x + before;
}

// Inclusive scan over the lanes of a warp.
__device__ __forceinline__ int64_t warp_scan(int64_t x) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The first (sequence, offset) of CTA `cta`'s run, and its end: fills sh and
// returns the tiles of the run (0: nothing to do).  All threads take part.
// Up to 32 sequences are a lane each: every warp finds the place by itself.
__device__ __forceinline__ int64_t division_start(const PagedArgs& c, const Division& v, int cta,
                                                  DivisionShared& sh) {
  if (c.B <= 32) {
    const int lane = threadIdx.x % 32;
    SeqInfo seq{0, 0};
    if (lane < c.B) seq = sequence(c, lane);
    const int64_t tiles = lane < c.B ? tiles_of(seq, v) * v.units : 0;
    const int64_t upto = warp_scan(tiles);
    const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
    const int64_t run = run_length(v, all);
    const int64_t begin = cta * run;
    if (begin >= upto - tiles && begin < upto) {
      // one lane of every warp: all write the same
      sh.b = lane;
      sh.seq = seq;
      sh.off = begin - (upto - tiles);
      sh.run = run;
    }
    if (cta == 0 && c.count && lane < c.B && c.lens[lane] >= 0 && c.count[lane] > c.T)
      flag_page(c.status);
    __syncthreads();
    return begin >= all ? 0 : min(run, all - begin);
  }
  const int per_thread = (c.B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(c.B, static_cast<int>(threadIdx.x) * per_thread);
  const int b1 = min(c.B, b0 + per_thread);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += seq_tiles(c, v, b);
    if (cta == 0 && c.count && c.lens[b] >= 0 && c.count[b] > c.T) flag_page(c.status);
  }
  int64_t at = block_scan(mine, sh) - mine;
  __syncthreads();
  const int64_t all = sh.total * v.units;
  const int64_t run = run_length(v, all);
  const int64_t begin = cta * run;
  if (begin < all && begin >= at * v.units && begin < (at + mine) * v.units) {
    for (int b = b0; b < b1; ++b) {
      const SeqInfo seq = sequence(c, b);
      const int64_t t = tiles_of(seq, v);
      if (begin < (at + t) * v.units) {
        sh.b = b;
        sh.seq = seq;
        sh.off = begin - at * v.units;
        sh.run = run;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  if (begin >= all) return 0;
  return min(run, all - begin);
}

// Tiles (of one unit) of the sequences before b, and of all.  All threads of
// the block take part.
__device__ __forceinline__ void division_before(const PagedArgs& c, const Division& v, int b,
                                                DivisionShared& sh, int64_t& ahead, int64_t& total) {
  if (c.B <= 32) {
    const int lane = threadIdx.x % 32;
    const int64_t upto = warp_scan(lane < c.B ? seq_tiles(c, v, lane) : 0);
    ahead = b > 0 ? __shfl_sync(0xffffffffu, upto, b - 1) : 0;
    total = __shfl_sync(0xffffffffu, upto, 31);
    return;
  }
  int64_t mine = 0, all = 0;
  for (int i = threadIdx.x; i < c.B; i += blockDim.x) {
    const int64_t t = seq_tiles(c, v, i);
    all += t;
    if (i < b) mine += t;
  }
  block_scan(mine, sh);
  __syncthreads();
  ahead = sh.total;
  __syncthreads();
  block_scan(all, sh);
  __syncthreads();
  total = sh.total;
}

// Walks a CTA's run unit by unit.
struct UnitWalk {
  int64_t left, off;  // tiles left in the run; offset within sequence b's tiles
  int b;
  // the present unit
  SeqInfo seq;
  int64_t tiles, first, last;  // of the unit; this CTA's part [first, last)
  int unit;

  __device__ void start(const PagedArgs& c, const Division& v, const DivisionShared& sh,
                        int64_t n) {
    left = n;
    b = sh.b;
    off = sh.off;
    if (left > 0) load(c, v);
  }
  // The same without a load: the sequence is the one that division_start found.
  __device__ void start_found(const Division& v, const DivisionShared& sh, int64_t n) {
    left = n;
    b = sh.b;
    off = sh.off;
    seq = sh.seq;
    if (left > 0) set(v);
  }
  __device__ bool done() const { return left <= 0; }
  __device__ void load(const PagedArgs& c, const Division& v) {
    seq = sequence(c, b);
    set(v);
  }
  __device__ void set(const Division& v) {
    tiles = tiles_of(seq, v);
    unit = static_cast<int>(off / tiles);
    first = off - unit * tiles;
    last = min(tiles, first + left);
  }
  __device__ void next(const PagedArgs& c, const Division& v) {
    left -= last - first;
    off += last - first;
    if (off == tiles * v.units) {
      ++b;
      off = 0;
    }
    if (left > 0) load(c, v);
  }
  __device__ bool whole() const { return first == 0 && last == tiles; }
  // Slot of a part that is not the whole unit.
  __device__ int slot(int cta) const { return 2 * cta + (first == 0 ? 1 : 0); }
};

}  // namespace ra
