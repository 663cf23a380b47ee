// Norm of every head of q and k with the position rotation, one pass over
// the rows, and its backward.
//
//   n = x w r,  r = 1 / sqrt(mean(x^2) + eps),  y = R(angle) n
//   dz = R(-angle) dy,  dx = r (dz w - x r^2 mean(dz w x)),  dw = sum dz x r
//
// Bound by memory: each element is read once and written once (the backward
// reads two).  A lane holds kP rotation pairs of a row: two pieces of kP
// elements, rot / 2 apart for the half-split pairing, adjacent for the
// interleaved one, so the rotation needs no exchange between lanes.  kP = 8
// (16-byte pieces of bf16) where d and rot are multiples of 16, else 4.  A row
// belongs to d / 2kP lanes, padded to a power of two for the row's sums.  A
// group of lanes stays with one token and walks over its heads: the angles
// of a lane are computed once per token, and the next heads are loaded,
// packed, before the present ones are worked on.  The arithmetic runs on
// pairs of floats (fma.rn.f32x2): with single ones the backward was bound by
// its instructions.
//
// pos * turns wraps modulo 2^64 as the angle does, and its upper half is the
// signed fraction of a turn.  turns is off by 2^-65 at most (2^-64 from 2^16
// radians on), so the angle is by |pos| 2^-65 turns beside fp32's own rounding
// of the fraction (2^-26): as good as fp32 can tell up to positions of 2^39.
//
// Measured, 32768 tokens of 32 + 8 heads of 128, bf16: forward 110 us (671 MB,
// 89 % of the copy rate; with 4-element pieces and one head ahead 219), backward
// 195 us (1007 MB, 76 %; single-float arithmetic 269, one head ahead 207).  The
// backward's rows need two sums that depend on one another, so it lives from
// the heads that are on their way: two at 128 registers with the weight in
// shared memory.  Three heads spill (217 us; 205 with the rotation in shared
// memory too), six through shared memory took 262, three blocks per SM spill.

#include <cuda_bf16.h>

#include "ra_paged.cuh"
#include "sm103_ptx.cuh"

namespace ra {
namespace {

using namespace ptx;

// Short blocks suit the forward (32768 tokens: 128 threads 110 us, 256 115, 64
// 113), long ones the backward, whose fixed blocks each take as many
// neighbouring tokens as they have groups (128 threads 214 us, 256 193).
constexpr int kForwardThreads = 128;
constexpr int kThreads = 256;

// Sum over the kLanes lanes of a row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A lane's part of a row as floats: the first and the second elements of its
// kP rotation pairs, two pairs to a register pair.
template <int kP>
struct Row {
  uint64_t p[kP / 2], q[kP / 2];
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int i = 0; i < kP / 2; ++i) p[i] = q[i] = pack_f32x2(x, x);
  }
  // Sum of products with another row's part.
  __device__ __forceinline__ float dot(const Row& o) const {
    uint64_t u = mul_f32x2(p[0], o.p[0]), v = mul_f32x2(q[0], o.q[0]);
#pragma unroll
    for (int i = 1; i < kP / 2; ++i) {
      u = fma_f32x2(p[i], o.p[i], u);
      v = fma_f32x2(q[i], o.q[i], v);
    }
    float a, b;
    unpack_f32x2(add_f32x2(u, v), a, b);
    return a + b;
  }
  __device__ __forceinline__ void scale(float x) {
    const uint64_t y = pack_f32x2(x, x);
#pragma unroll
    for (int i = 0; i < kP / 2; ++i) {
      p[i] = mul_f32x2(p[i], y);
      q[i] = mul_f32x2(q[i], y);
    }
  }
  __device__ __forceinline__ void times(const Row& o) {
#pragma unroll
    for (int i = 0; i < kP / 2; ++i) {
      p[i] = mul_f32x2(p[i], o.p[i]);
      q[i] = mul_f32x2(q[i], o.q[i]);
    }
  }
  // this += a * b
  __device__ __forceinline__ void add_product(const Row& a, const Row& b) {
#pragma unroll
    for (int i = 0; i < kP / 2; ++i) {
      p[i] = fma_f32x2(a.p[i], b.p[i], p[i]);
      q[i] = fma_f32x2(a.q[i], b.q[i], q[i]);
    }
  }
  // this += a * x
  __device__ __forceinline__ void add_scaled(const Row& a, float x) {
    const uint64_t y = pack_f32x2(x, x);
#pragma unroll
    for (int i = 0; i < kP / 2; ++i) {
      p[i] = fma_f32x2(a.p[i], y, p[i]);
      q[i] = fma_f32x2(a.q[i], y, q[i]);
    }
  }
};

// A lane's two pieces of a row, as they lie in memory.
template <typename E, int kP, bool kInterleaved>
struct Pieces {
  Packed<E, kP> lo, hi;
  __device__ __forceinline__ void zero() {
    lo.zero();
    hi.zero();
  }
  __device__ __forceinline__ void load(const E* p, int o1, int o2) {
    lo.load(p + o1);
    hi.load(p + o2);
  }
  __device__ __forceinline__ void get(Row<kP>& r) const {
    float x[kP], y[kP];
    lo.get(x);
    hi.get(y);
#pragma unroll
    for (int i = 0; i < kP / 2; ++i) {
      if (kInterleaved) {  // elements p0 q0 p1 q1 ... through both pieces
        const float* z = 4 * i < kP ? x + 4 * i : y + 4 * i - kP;
        r.p[i] = pack_f32x2(z[0], z[2]);
        r.q[i] = pack_f32x2(z[1], z[3]);
      } else {
        r.p[i] = pack_f32x2(x[2 * i], x[2 * i + 1]);
        r.q[i] = pack_f32x2(y[2 * i], y[2 * i + 1]);
      }
    }
  }
};

// The floats of a part in the order of its two pieces.
template <int kP, bool kInterleaved>
__device__ __forceinline__ void in_order(const Row<kP>& r, float (&x)[kP], float (&y)[kP]) {
#pragma unroll
  for (int i = 0; i < kP / 2; ++i) {
    if (kInterleaved) {
      float* z = 4 * i < kP ? x + 4 * i : y + 4 * i - kP;
      unpack_f32x2(r.p[i], z[0], z[2]);
      unpack_f32x2(r.q[i], z[1], z[3]);
    } else {
      unpack_f32x2(r.p[i], x[2 * i], x[2 * i + 1]);
      unpack_f32x2(r.q[i], y[2 * i], y[2 * i + 1]);
    }
  }
}

template <typename E, int kP, bool kInterleaved>
__device__ __forceinline__ void store_pieces(E* p, int o1, int o2, const Row<kP>& r) {
  float x[kP], y[kP];
  in_order<kP, kInterleaved>(r, x, y);
  Packed<E, kP> w;
  w.set(x);
  w.store(p + o1);
  w.set(y);
  w.store(p + o2);
}

// One lane's place in a row: the offsets of its two pieces and the
// rotations of its pairs for one token.
template <int kP>
struct LanePlace {
  int o1, o2;
  bool live, rotated;
  uint64_t c[kP / 2], s[kP / 2];

  __device__ void place(int l, int d, int rot, bool interleaved) {
    live = 2 * kP * l < d;
    rotated = 2 * kP * l < rot;
    if (rotated && !interleaved) {
      o1 = kP * l;
      o2 = rot / 2 + kP * l;
    } else {
      o1 = live ? 2 * kP * l : 0;
      o2 = o1 + kP;
    }
  }
  // sign -1: rotates back.
  __device__ void angles(const NormArgs& a, int l, int64_t token, float sign) {
    if (!rotated) return;
    float cs[kP], sn[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int64_t pos = a.positions[a.rope.axis[kP * l + i] * a.tokens + token];
      const uint64_t turn = static_cast<uint64_t>(pos) * a.rope.turns[kP * l + i];
      const int32_t frac = static_cast<int32_t>(turn >> 32);  // turns * 2^32, signed
      sincospif(static_cast<float>(frac) * 0x1p-31f, &sn[i], &cs[i]);
    }
#pragma unroll
    for (int i = 0; i < kP / 2; ++i) {
      c[i] = pack_f32x2(cs[2 * i], cs[2 * i + 1]);
      s[i] = pack_f32x2(sign * sn[2 * i], sign * sn[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void rotate(Row<kP>& r) const {
    const uint64_t minus = pack_f32x2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < kP / 2; ++i) {
      const uint64_t qs = mul_f32x2(r.q[i], s[i]);
      const uint64_t qc = mul_f32x2(r.q[i], c[i]);
      const uint64_t p = r.p[i];
      r.p[i] = fma_f32x2(p, c[i], mul_f32x2(qs, minus));
      r.q[i] = fma_f32x2(p, s[i], qc);
    }
  }
};

template <typename E, int kP, bool kInterleaved>
__device__ __forceinline__ void load_weight(const NormSide& s, const LanePlace<kP>& lp, Row<kP>& w) {
  w.fill(1.f);
  if (s.weight && lp.live) {
    Pieces<E, kP, kInterleaved> x;
    x.load(static_cast<const E*>(s.weight), lp.o1, lp.o2);
    x.get(w);
  }
}

// blockIdx.x: tokens; blockIdx.y: a run of `run` heads of q's, then k's.
template <typename E, int kP, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kForwardThreads) norm_rope_kernel(const __grid_constant__ NormArgs a,
                                                             int run) {
  constexpr int kAhead = 4;
  const int l = threadIdx.x % kLanes;
  const int64_t token =
      static_cast<int64_t>(blockIdx.x) * (kForwardThreads / kLanes) + threadIdx.x / kLanes;
  const bool here = token < a.tokens;
  const int64_t b = here ? token / a.N : 0, n = here ? token % a.N : 0;
  LanePlace<kP> lp;
  lp.place(l, a.d, a.has_rope ? a.rope.rot : 0, kInterleaved);
  const bool live = lp.live && here;
  const float inv_d = 1.f / a.d;
  const int hq = a.side[0].heads;
  const int h_begin = blockIdx.y * run, h_end = min(hq + a.side[1].heads, h_begin + run);
  const E* src[2];
  E* dst[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    src[t] = static_cast<const E*>(a.side[t].x) + b * a.side[t].xs.b + n * a.side[t].xs.n;
    dst[t] = static_cast<E*>(a.side[t].y) + b * a.side[t].ys.b + n * a.side[t].ys.n;
  }
  Pieces<E, kP, kInterleaved> next[kAhead];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = h0 + j;
      next[j].zero();
      if (h < h_end && live)
        next[j].load(h < hq ? src[0] + h * a.side[0].xs.h : src[1] + (h - hq) * a.side[1].xs.h, lp.o1,
                     lp.o2);
    }
  };
  fetch(h_begin);
  lp.angles(a, l, here ? token : 0, 1.f);
  Row<kP> w;
  int loaded = -1;
  for (int h0 = h_begin; h0 < h_end; h0 += kAhead) {
    Pieces<E, kP, kInterleaved> now[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) now[j] = next[j];
    if (h0 + kAhead < h_end) fetch(h0 + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = h0 + j;
      if (h >= h_end) break;
      const int side = h >= hq;
      Row<kP> x;
      now[j].get(x);
      if (a.eps >= 0.f) {
        if (side != loaded) {
          load_weight<E, kP, kInterleaved>(a.side[side], lp, w);
          loaded = side;
        }
        x.scale(rsqrtf(row_sum<kLanes>(x.dot(x)) * inv_d + a.eps));
        x.times(w);
      }
      if (lp.rotated) lp.rotate(x);
      if (live)
        store_pieces<E, kP, kInterleaved>(
            side ? dst[1] + (h - hq) * a.side[1].ys.h : dst[0] + h * a.side[0].ys.h, lp.o1, lp.o2, x);
    }
  }
}

// A fixed grid, two blocks per SM, walks over (token tile, run of heads)
// items of one side and then of the other with dw in registers; block sums go
// to a.partial, one row per block and side.
template <typename E, int kP, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 2)
    norm_rope_backward_kernel(const __grid_constant__ NormArgs a, int run, int64_t tiles) {
  constexpr int kGroups = kThreads / kLanes;
  constexpr int kAhead = 2;
  __shared__ float sums[kGroups][kLanes * 2 * kP + 4];
  __shared__ ulonglong2 weight[kP / 2][kLanes];  // in shared memory, not in registers
  const int l = threadIdx.x % kLanes;
  const int group = threadIdx.x / kLanes;
  const float inv_d = 1.f / a.d;
  LanePlace<kP> lp;
  lp.place(l, a.d, a.has_rope ? a.rope.rot : 0, kInterleaved);
  for (int t = 0; t < 2; ++t) {
    const NormSide& s = a.side[t];
    Row<kP> dw;
    dw.fill(0.f);
    __syncthreads();
    if (group == 0) {
      Row<kP> w;
      load_weight<E, kP, kInterleaved>(s, lp, w);
#pragma unroll
      for (int i = 0; i < kP / 4; ++i) {
        weight[i][l] = make_ulonglong2(w.p[2 * i], w.p[2 * i + 1]);
        weight[kP / 4 + i][l] = make_ulonglong2(w.q[2 * i], w.q[2 * i + 1]);
      }
    }
    __syncthreads();
    const int runs = (s.heads + run - 1) / run;
    for (int64_t item = blockIdx.x; item < tiles * runs; item += gridDim.x) {
      const int64_t token = (item / runs) * kGroups + group;
      const int h_begin = static_cast<int>(item % runs) * run;
      const int h_end = min(s.heads, h_begin + run);
      const bool here = token < a.tokens;
      const int64_t b = here ? token / a.N : 0, n = here ? token % a.N : 0;
      const bool live = lp.live && here;
      // A group without a token adds zeros to dw; with eps = 0 they would be 0 * inf.
      const float eps = here ? a.eps : 1.f;
      const E* src = static_cast<const E*>(s.x) + b * s.xs.b + n * s.xs.n;
      const E* dy = static_cast<const E*>(s.dy) + (b * s.heads * a.N + n) * a.d;
      E* dst = static_cast<E*>(s.y) + b * s.ys.b + n * s.ys.n;
      Pieces<E, kP, kInterleaved> next_x[kAhead], next_g[kAhead];
      auto fetch = [&](int h, int j) {
        next_x[j].zero();
        next_g[j].zero();
        if (live && h < h_end) {
          next_g[j].load(dy + static_cast<int64_t>(h) * a.N * a.d, lp.o1, lp.o2);
          if (a.eps >= 0.f) next_x[j].load(src + h * s.xs.h, lp.o1, lp.o2);
        }
      };
#pragma unroll
      for (int j = 0; j < kAhead; ++j) fetch(h_begin + j, j);
      lp.angles(a, l, here ? token : 0, -1.f);
      for (int h0 = h_begin; h0 < h_end; h0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int h = h0 + j;
          if (h >= h_end) break;
          Row<kP> g, x;
          next_g[j].get(g);
          next_x[j].get(x);
          fetch(h + kAhead, j);
          if (lp.rotated) lp.rotate(g);
          if (a.eps >= 0.f) {
            const float r = rsqrtf(row_sum<kLanes>(x.dot(x)) * inv_d + eps);
            x.scale(r);  // the normalised row
            dw.add_product(g, x);
#pragma unroll
            for (int i = 0; i < kP / 4; ++i) {
              const ulonglong2 wp = weight[i][l], wq = weight[kP / 4 + i][l];
              g.p[2 * i] = mul_f32x2(g.p[2 * i], wp.x);
              g.p[2 * i + 1] = mul_f32x2(g.p[2 * i + 1], wp.y);
              g.q[2 * i] = mul_f32x2(g.q[2 * i], wq.x);
              g.q[2 * i + 1] = mul_f32x2(g.q[2 * i + 1], wq.y);
            }
            const float mean = row_sum<kLanes>(g.dot(x)) * inv_d;
            g.add_scaled(x, -mean);
            g.scale(r);
          }
          if (live) store_pieces<E, kP, kInterleaved>(dst + h * s.ys.h, lp.o1, lp.o2, g);
        }
      }
    }
    if (!a.partial) continue;
    __syncthreads();
    if (lp.live) {
      float x[kP], y[kP];
      in_order<kP, kInterleaved>(dw, x, y);
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        sums[group][lp.o1 + i] = x[i];
        sums[group][lp.o2 + i] = y[i];
      }
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

// Heads per run: all of a token's heads while that makes `blocks` blocks per
// SM, else fewer: short blocks even the end of the launch, and a decode
// step's few tokens spread out.  16 for the forward; 1 for the backward, whose
// items load nothing ahead of one another, so that longer runs pay more than
// an even end (32 + 8 heads of 128, us at 1 and 16: 300 tokens 16.6 20.6, 1560
// 28.8 32.9, 6000 53.4 51.4, 9000 63.6 72.7; 8 + 2 heads: 3000 tokens 20.7 24.6,
// 16000 41.1 47.3).
int heads_per_run(int64_t token_tiles, int heads, int blocks) {
  const int64_t want = static_cast<int64_t>(device_sm_count()) * blocks;
  int64_t runs = (want + token_tiles - 1) / token_tiles;
  if (runs > heads) runs = heads;
  return static_cast<int>((heads + runs - 1) / runs);
}

template <typename E, int kP, int kLanes>
cudaError_t launch_t(const NormArgs& a, bool backward, cudaStream_t s) {
  const int heads = a.side[0].heads + a.side[1].heads;
  const int groups = (backward ? kThreads : kForwardThreads) / kLanes;
  const int64_t tiles = (a.tokens + groups - 1) / groups;
  const int run = heads_per_run(tiles, heads, backward ? 1 : 16);
  const bool inter = a.has_rope && a.rope.interleaved;
  if (!backward) {
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((heads + run - 1) / run));
    if (inter)
      norm_rope_kernel<E, kP, kLanes, true><<<grid, kForwardThreads, 0, s>>>(a, run);
    else
      norm_rope_kernel<E, kP, kLanes, false><<<grid, kForwardThreads, 0, s>>>(a, run);
    return cudaGetLastError();
  }
  const int most = a.side[0].heads > a.side[1].heads ? a.side[0].heads : a.side[1].heads;
  const int64_t items = tiles * ((most + run - 1) / run);
  const int blocks = static_cast<int>(items < kNormBackwardBlocks ? items : kNormBackwardBlocks);
  if (inter)
    norm_rope_backward_kernel<E, kP, kLanes, true><<<blocks, kThreads, 0, s>>>(a, run, tiles);
  else
    norm_rope_backward_kernel<E, kP, kLanes, false><<<blocks, kThreads, 0, s>>>(a, run, tiles);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  norm_weight_kernel<<<dim3((a.d + 31) / 32, 2), 256, 0, s>>>(
      a.partial, a.side[0].dweight, a.side[1].dweight, a.d, blocks);
  return cudaGetLastError();
}

template <typename E, int kP>
cudaError_t by_width(const NormArgs& a, bool backward, cudaStream_t s) {
  const int lanes = a.d / (2 * kP);
  if (lanes <= 1) return launch_t<E, kP, 1>(a, backward, s);
  if (lanes <= 2) return launch_t<E, kP, 2>(a, backward, s);
  if (lanes <= 4) return launch_t<E, kP, 4>(a, backward, s);
  if (lanes <= 8) return launch_t<E, kP, 8>(a, backward, s);
  if (lanes <= 16) return launch_t<E, kP, 16>(a, backward, s);
  return launch_t<E, kP, 32>(a, backward, s);
}

// Pieces of 16 bytes where the widths and every address allow them.
bool wide(const NormArgs& a) {
  if (a.d % 16 != 0 || (a.has_rope && a.rope.rot % 16 != 0)) return false;
  for (const NormSide& s : a.side) {
    uintptr_t bits = 0;
    for (const void* p : {s.x, s.dy, static_cast<const void*>(s.y), s.weight})
      bits |= reinterpret_cast<uintptr_t>(p);
    for (const Strides& st : {s.xs, s.ys}) bits |= static_cast<uintptr_t>(2 * (st.b | st.h | st.n));
    if (bits % 16 != 0) return false;
  }
  return true;
}

cudaError_t dispatch(const NormArgs& a, bool bf16, bool backward, cudaStream_t s) {
  if (!bf16) return by_width<float, 4>(a, backward, s);
  return wide(a) ? by_width<__nv_bfloat16, 8>(a, backward, s)
                 : by_width<__nv_bfloat16, 4>(a, backward, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormArgs& a, bool bf16, cudaStream_t s) {
  return dispatch(a, bf16, false, s);
}

cudaError_t launch_norm_rope_backward(const NormArgs& a, bool bf16, cudaStream_t s) {
  return dispatch(a, bf16, true, s);
}

}  // namespace ra
