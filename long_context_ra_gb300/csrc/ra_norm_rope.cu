// Norm of every head of q and k with the position rotation, one pass over
// the rows, and its backward.
//
//   n = x w r,  r = 1 / sqrt(mean(x^2) + eps),  y = R(angle) n
//   dz = R(-angle) dy,  dx = r (dz w - x r^2 mean(dz w x)),  dw = sum dz x r
//
// Bound by memory: each element is read once and written once (the backward
// reads two).  A row of d elements belongs to d / 8 lanes of a warp, padded
// to a power of two for the row's sums.  A lane holds the 8 elements of four
// rotation pairs: two 4-element pieces, rot / 2 apart for the half-split
// pairing, adjacent for the interleaved one, so the rotation needs no
// exchange between lanes.  A group of lanes stays with one token and walks
// over its heads: the four angles of a lane are computed once per token, and
// the loads of several heads are in flight together.
//
// The angle is exact for any position: pos * turns wraps modulo 2^64 and its
// upper half is the signed fraction of a turn.

#include <cuda_bf16.h>

#include "ra_internal.h"
#include "ra_serve.h"

namespace ra {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load4(const float* p, float* r) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  r[0] = x.x;
  r[1] = x.y;
  r[2] = x.z;
  r[3] = x.w;
}

__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* r) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  r[0] = __uint_as_float(x.x << 16);
  r[1] = __uint_as_float(x.x & 0xffff0000u);
  r[2] = __uint_as_float(x.y << 16);
  r[3] = __uint_as_float(x.y & 0xffff0000u);
}

__device__ __forceinline__ void store4(float* p, const float* r) {
  *reinterpret_cast<float4*>(p) = make_float4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* r) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(r[0], r[1]);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(r[2], r[3]);
  uint2 x;
  x.x = *reinterpret_cast<const uint32_t*>(&lo);
  x.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p) = x;
}

// Sum over the kLanes lanes of a row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// One lane's place in a row: the offsets of its two pieces and the
// rotations of its pairs for one token (cosine 1, sine 0 past rot).
struct LanePlace {
  int o1, o2;
  bool live, rotated;
  float c[4], s[4];

  __device__ void place(int l, int d, int rot, bool interleaved) {
    live = 8 * l < d;
    rotated = 8 * l < rot;
    if (rotated && !interleaved) {
      o1 = 4 * l;
      o2 = rot / 2 + 4 * l;
    } else {
      o1 = live ? 8 * l : 0;
      o2 = o1 + 4;
    }
  }
  __device__ void angles(const NormArgs& a, int l, int64_t token) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
    }
    if (!rotated) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t pos = a.positions[a.rope.axis[4 * l + i] * a.tokens + token];
      const uint64_t turn = static_cast<uint64_t>(pos) * a.rope.turns[4 * l + i];
      const int32_t frac = static_cast<int32_t>(turn >> 32);  // turns * 2^32, signed
      sincospif(static_cast<float>(frac) * 0x1p-31f, &s[i], &c[i]);
    }
  }
  // x[0..3] at o1, x[4..7] at o2; sign -1 rotates back.
  __device__ void rotate(float* x, bool interleaved, float sign) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float si = sign * s[i];
      float& p = interleaved ? x[2 * i] : x[i];
      float& q = interleaved ? x[2 * i + 1] : x[i + 4];
      const float u = p * c[i] - q * si;
      q = q * c[i] + p * si;
      p = u;
    }
  }
};

template <typename E>
__device__ __forceinline__ void load_weight(const NormSide& s, const LanePlace& lp, float* w) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (s.weight && lp.live) {
    load4(static_cast<const E*>(s.weight) + lp.o1, w);
    load4(static_cast<const E*>(s.weight) + lp.o2, w + 4);
  }
}

// blockIdx.x: tokens; blockIdx.y: a run of `run` heads of q's, then k's.
template <typename E, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormArgs a,
                                                             int run) {
  const int l = threadIdx.x % kLanes;
  const int64_t token =
      static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const bool here = token < a.tokens;
  const int64_t b = here ? token / a.N : 0, n = here ? token % a.N : 0;
  LanePlace lp;
  lp.place(l, a.d, a.has_rope ? a.rope.rot : 0, kInterleaved);
  const bool live = lp.live && here;
  lp.angles(a, l, here ? token : 0);
  const int total = a.side[0].heads + a.side[1].heads;
  const int h_end = min(total, static_cast<int>(blockIdx.y + 1) * run);
  float w[8];
  int loaded = -1;
  constexpr int kAhead = 4;
  for (int h0 = blockIdx.y * run; h0 < h_end; h0 += kAhead) {
    float x[kAhead][8];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = h0 + j;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
      if (h < h_end && live) {
        const NormSide& s = a.side[h >= a.side[0].heads];
        const int hh = h >= a.side[0].heads ? h - a.side[0].heads : h;
        const E* p = static_cast<const E*>(s.x) + b * s.xs.b + hh * s.xs.h + n * s.xs.n;
        load4(p + lp.o1, x[j]);
        load4(p + lp.o2, x[j] + 4);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = h0 + j;
      if (h >= h_end) break;
      const int side = h >= a.side[0].heads;
      const NormSide& s = a.side[side];
      if (side != loaded) {
        load_weight<E>(s, lp, w);
        loaded = side;
      }
      if (a.eps >= 0.f) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[j][i], x[j][i], ss);
        const float r = rsqrtf(row_sum<kLanes>(ss) / a.d + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = x[j][i] * r * w[i];
      }
      if (lp.rotated) lp.rotate(x[j], kInterleaved, 1.f);
      if (live) {
        const int hh = side ? h - a.side[0].heads : h;
        E* p = static_cast<E*>(s.y) + b * s.ys.b + hh * s.ys.h + n * s.ys.n;
        store4(p + lp.o1, x[j]);
        store4(p + lp.o2, x[j] + 4);
      }
    }
  }
}

// A fixed grid walks over (token tile, run of heads) items and keeps dw of
// both sides in registers; block sums go to a.partial, one row per block.
template <typename E, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
    norm_rope_backward_kernel(const __grid_constant__ NormArgs a, int run, int runs,
                              int64_t items) {
  constexpr int kGroups = kThreads / kLanes;
  __shared__ float sums[kGroups][kLanes * 8 + 4];
  const int l = threadIdx.x % kLanes;
  const int group = threadIdx.x / kLanes;
  LanePlace lp;
  lp.place(l, a.d, a.has_rope ? a.rope.rot : 0, kInterleaved);
  const int total = a.side[0].heads + a.side[1].heads;
  float dw[2][8], w[2][8];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    load_weight<E>(a.side[t], lp, w[t]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[t][i] = 0.f;
  }
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t token = (item / runs) * kGroups + group;
    const int h_begin = static_cast<int>(item % runs) * run;
    const int h_end = min(total, h_begin + run);
    const bool here = token < a.tokens;
    const int64_t b = here ? token / a.N : 0, n = here ? token % a.N : 0;
    const bool live = lp.live && here;
    lp.angles(a, l, here ? token : 0);
    constexpr int kAhead = 2;
    for (int h0 = h_begin; h0 < h_end; h0 += kAhead) {
      float x[kAhead][8], g[kAhead][8];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int h = h0 + j;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = g[j][i] = 0.f;
        if (h < h_end && live) {
          const NormSide& s = a.side[h >= a.side[0].heads];
          const int hh = h >= a.side[0].heads ? h - a.side[0].heads : h;
          const E* gy = static_cast<const E*>(s.dy) + ((b * s.heads + hh) * a.N + n) * a.d;
          load4(gy + lp.o1, g[j]);
          load4(gy + lp.o2, g[j] + 4);
          if (a.eps >= 0.f) {
            const E* p = static_cast<const E*>(s.x) + b * s.xs.b + hh * s.xs.h + n * s.xs.n;
            load4(p + lp.o1, x[j]);
            load4(p + lp.o2, x[j] + 4);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int h = h0 + j;
        if (h >= h_end) break;
        const int side = h >= a.side[0].heads;
        const NormSide& s = a.side[side];
        if (lp.rotated) lp.rotate(g[j], kInterleaved, -1.f);
        if (a.eps >= 0.f) {
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[j][i], x[j][i], ss);
          const float r = rsqrtf(row_sum<kLanes>(ss) / a.d + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float n = x[j][i] * r;  // the normalised row
            const float t = g[j][i] * n;
            x[j][i] = n;
            if (side)
              dw[1][i] += t;
            else
              dw[0][i] += t;
            g[j][i] *= side ? w[1][i] : w[0][i];
            dot = fmaf(g[j][i], n, dot);
          }
          const float mean = row_sum<kLanes>(dot) / a.d;
#pragma unroll
          for (int i = 0; i < 8; ++i) g[j][i] = r * (g[j][i] - x[j][i] * mean);
        }
        if (live) {
          const int hh = side ? h - a.side[0].heads : h;
          E* p = static_cast<E*>(s.y) + b * s.ys.b + hh * s.ys.h + n * s.ys.n;
          store4(p + lp.o1, g[j]);
          store4(p + lp.o2, g[j] + 4);
        }
      }
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    __syncthreads();
    if (lp.live) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[group][i < 4 ? lp.o1 + i : lp.o2 + i - 4] = dw[t][i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.d; e += kThreads) {
      float x = 0.f;
      for (int gr = 0; gr < kGroups; ++gr) x += sums[gr][e];
      a.partial[(static_cast<int64_t>(blockIdx.x) * 2 + t) * a.d + e] = x;
    }
  }
}

// dw = the sum of the blocks' rows, in a fixed order; 64-bit sums cost
// nothing here.  32 columns per block, 8 threads per column.
__global__ void __launch_bounds__(256) norm_weight_kernel(const float* partial, float* dwq,
                                                          float* dwk, int d, int blocks) {
  __shared__ double part[8][32];
  const int lane = threadIdx.x % 32, row = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + lane;
  float* dst = blockIdx.y ? dwk : dwq;
  if (!dst) return;
  double x = 0;
  if (col < d)
    for (int i = row; i < blocks; i += 8)
      x += partial[(static_cast<int64_t>(i) * 2 + blockIdx.y) * d + col];
  part[row][lane] = x;
  __syncthreads();
  if (row == 0 && col < d) {
    for (int i = 1; i < 8; ++i) x += part[i][lane];
    dst[col] = static_cast<float>(x);
  }
}

// Heads per run: all of a token's heads while that fills the GPU's SMs four
// times over, else fewer, so that a decode step's few tokens spread out.
int heads_per_run(int64_t token_tiles, int heads) {
  const int64_t want = static_cast<int64_t>(device_sm_count()) * 4;
  int64_t runs = (want + token_tiles - 1) / token_tiles;
  if (runs > heads) runs = heads;
  return static_cast<int>((heads + runs - 1) / runs);
}

template <typename E, int kLanes>
cudaError_t forward_t(const NormArgs& a, cudaStream_t s) {
  const int heads = a.side[0].heads + a.side[1].heads;
  constexpr int kGroups = kThreads / kLanes;
  const int64_t tiles = (a.tokens + kGroups - 1) / kGroups;
  const int run = heads_per_run(tiles, heads);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((heads + run - 1) / run));
  if (a.has_rope && a.rope.interleaved)
    norm_rope_kernel<E, kLanes, true><<<grid, kThreads, 0, s>>>(a, run);
  else
    norm_rope_kernel<E, kLanes, false><<<grid, kThreads, 0, s>>>(a, run);
  return cudaGetLastError();
}

template <typename E, int kLanes>
cudaError_t backward_t(const NormArgs& a, cudaStream_t s) {
  const int heads = a.side[0].heads + a.side[1].heads;
  constexpr int kGroups = kThreads / kLanes;
  const int64_t tiles = (a.tokens + kGroups - 1) / kGroups;
  const int run = heads_per_run(tiles, heads);
  const int runs = (heads + run - 1) / run;
  const int64_t items = tiles * runs;
  const int blocks = static_cast<int>(items < kNormBackwardBlocks ? items : kNormBackwardBlocks);
  if (a.has_rope && a.rope.interleaved)
    norm_rope_backward_kernel<E, kLanes, true><<<blocks, kThreads, 0, s>>>(a, run, runs, items);
  else
    norm_rope_backward_kernel<E, kLanes, false><<<blocks, kThreads, 0, s>>>(a, run, runs, items);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  norm_weight_kernel<<<dim3((a.d + 31) / 32, 2), 256, 0, s>>>(
      a.partial, a.side[0].dweight, a.side[1].dweight, a.d, blocks);
  return cudaGetLastError();
}

template <typename E>
cudaError_t dispatch(const NormArgs& a, bool backward, cudaStream_t s) {
  if (a.d <= 16) return backward ? backward_t<E, 2>(a, s) : forward_t<E, 2>(a, s);
  if (a.d <= 32) return backward ? backward_t<E, 4>(a, s) : forward_t<E, 4>(a, s);
  if (a.d <= 64) return backward ? backward_t<E, 8>(a, s) : forward_t<E, 8>(a, s);
  if (a.d <= 128) return backward ? backward_t<E, 16>(a, s) : forward_t<E, 16>(a, s);
  return backward ? backward_t<E, 32>(a, s) : forward_t<E, 32>(a, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? dispatch<__nv_bfloat16>(a, false, s) : dispatch<float>(a, false, s);
}

cudaError_t launch_norm_rope_backward(const NormArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? dispatch<__nv_bfloat16>(a, true, s) : dispatch<float>(a, true, s);
}

}  // namespace ra
