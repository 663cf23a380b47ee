// Writing new tokens into a paged K/V cache (quantising them for an 8-bit
// one) and reading positions back.
//
// Bound by memory: every element crosses once.  A row of d elements belongs
// to d / kV lanes (padded to a power of two for the row's maximum).  A group
// of lanes takes one token, finds its page once and walks over a run of the
// 2 x heads rows of K and V; the next rows are loaded, packed, before the
// present ones are worked on.  Neighbouring groups hold neighbouring tokens,
// whose rows lie next to each other in a page.
//
// Writes take 16 elements a lane (8-bit rows of 128 then are 16-byte pieces; 8
// elements: 90 us instead of 66 for 53k tokens of 8 heads) and two rows ahead
// (four: 69).  Reads take 8 (16: 154 us instead of 125 for 131072 positions of
// 8 heads out of 8 bits; a lane then stores 32 bytes in two instructions, each
// of which fills half of a line) and four rows ahead (eight: 127, two: 140).
// Both choices were measured with bf16 rows and an 8-bit cache.  With the others
// a lane moves 32 or 64 bytes in steps of 16, in half lines; one sequence, 8
// heads of 128, us by graph replay and the bytes' floor:
//   53248 written   bf16 to 8 bits 53 (48), to bf16 75 (64); f32 to 8 bits 89
//                   (80), to f32 158 (128)
//   131072 read     8 bits to bf16 123 (119), bf16 160 (158); 8 bits to f32 265
//                   (198), f32 341 (316)

#include "ra_paged.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
template <int kLanes>
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

template <typename E, typename H>
struct Same {
  static constexpr bool value = false;
};
template <typename E>
struct Same<E, E> {
  static constexpr bool value = true;
};

template <typename E, typename H, int kV, int kLanes>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheCopyArgs a,
                                                               int run) {
  constexpr bool k8 = !Same<E, H>::value;
  constexpr int kAhead = 2;
  const PagedArgs& c = a.c;
  const int l = threadIdx.x % kLanes;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int b = static_cast<int>(min(token / c.T, static_cast<int64_t>(c.B)));
  const int t = static_cast<int>(token % c.T);
  int64_t base = -1;
  if (b < c.B) {
    const SeqInfo s = sequence(c, b);
    if (t < s.cnt) base = cache_row(c, b, s.len + t);
    if (t == 0 && c.count && c.lens[b] >= 0 && c.count[b] > c.T) flag_page(c.status);
  }
  const bool live = base >= 0 && kV * l < c.d;
  const int r_begin = blockIdx.y * run, r_end = min(2 * c.heads, r_begin + run);
  const E* src_k = static_cast<const E*>(a.k) + b * a.ks.b + t * a.ks.n + kV * l;
  const E* src_v = static_cast<const E*>(a.v) + b * a.vs.b + t * a.vs.n + kV * l;
  Packed<E, kV> next[kAhead];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = r0 + j;
      next[j].zero();
      if (r < r_end && live)
        next[j].load(r < c.heads ? src_k + r * a.ks.h : src_v + (r - c.heads) * a.vs.h);
    }
  };
  fetch(r_begin);
  for (int r0 = r_begin; r0 < r_end; r0 += kAhead) {
    Packed<E, kV> now[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) now[j] = next[j];
    if (r0 + kAhead < r_end) fetch(r0 + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = r0 + j;
      if (r >= r_end) break;
      const bool v = r >= c.heads;
      const int64_t row = base + (static_cast<int64_t>(v ? r - c.heads : r) << c.page_shift);
      if (k8) {
        float x[kV];
        now[j].get(x);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const float y = fabsf(x[i]);
          m = y < INFINITY ? fmaxf(m, y) : m;  // finite elements only
        }
        const uint32_t e = row_exponent(row_max<kLanes>(m));
        const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] *= inv;
        if (live) {
          Packed<H, kV> out;
          out.set(x);
          out.store(static_cast<uint8_t*>(v ? c.v : c.k) + row * c.d + kV * l);
          if (l == 0) (v ? c.ve : c.ke)[row] = static_cast<uint8_t>(e);
        }
      } else if (live) {
        now[j].store(static_cast<E*>(v ? c.v : c.k) + row * c.d + kV * l);
      }
    }
  }
}

template <typename E, typename H, int kV, int kLanes>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheCopyArgs a,
                                                              int run) {
  constexpr bool k8 = !Same<E, H>::value;
  constexpr int kAhead = 4;
  const PagedArgs& c = a.c;
  const int l = threadIdx.x % kLanes;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (token >= c.B * a.n || kV * l >= c.d) return;
  const int b = static_cast<int>(token / a.n);
  const int64_t n = token % a.n;
  const int64_t base = a.first + n < c.lens[b] ? cache_row(c, b, a.first + n) : -1;
  const int r_begin = blockIdx.y * run, r_end = min(2 * c.heads, r_begin + run);
  Packed<H, kV> next[kAhead];
  uint32_t next_e[kAhead];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = r0 + j;
      next[j].zero();
      next_e[j] = 127;
      if (r < r_end && base >= 0) {
        const bool v = r >= c.heads;
        const int64_t row = base + (static_cast<int64_t>(v ? r - c.heads : r) << c.page_shift);
        next[j].load(static_cast<const H*>(v ? c.v : c.k) + row * c.d + kV * l);
        if (k8) next_e[j] = (v ? c.ve : c.ke)[row];
      }
    }
  };
  fetch(r_begin);
  for (int r0 = r_begin; r0 < r_end; r0 += kAhead) {
    Packed<H, kV> now[kAhead];
    uint32_t e[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      now[j] = next[j];
      e[j] = next_e[j];
    }
    if (r0 + kAhead < r_end) fetch(r0 + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = r0 + j;
      if (r >= r_end) break;
      const bool v = r >= c.heads;
      const int h = v ? r - c.heads : r;
      E* p = static_cast<E*>(v ? a.v : a.k) + ((static_cast<int64_t>(b) * c.heads + h) * a.n + n) * c.d +
             kV * l;
      if (k8) {
        float x[kV];
        now[j].get(x);
        const float sc = exp_scale(e[j]);
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] *= sc;
        Packed<E, kV> out;
        out.set(x);
        out.store(p);
      } else {
        now[j].store(p);
      }
    }
  }
}

// Rows per run: all 2 x heads of a token while that makes eight blocks per
// SM, else fewer: short blocks even the end of the launch, and a decode
// step's few tokens spread out.
int rows_per_run(int64_t tiles, int rows) {
  const int64_t want = static_cast<int64_t>(device_sm_count()) * 8;
  int64_t runs = (want + tiles - 1) / tiles;
  if (runs > rows) runs = rows;
  return static_cast<int>((rows + runs - 1) / runs);
}

template <typename E, typename H, int kV, int kLanes>
cudaError_t launch_t(const CacheCopyArgs& a, bool write, cudaStream_t s) {
  const int64_t tokens = a.c.B * (write ? static_cast<int64_t>(a.c.T) : a.n);
  constexpr int kGroups = kThreads / kLanes;
  const int64_t tiles = (tokens + kGroups - 1) / kGroups;
  const int rows = 2 * a.c.heads;
  const int run = rows_per_run(tiles, rows);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((rows + run - 1) / run));
  if (write)
    cache_write_kernel<E, H, kV, kLanes><<<grid, kThreads, 0, s>>>(a, run);
  else
    cache_read_kernel<E, H, kV, kLanes><<<grid, kThreads, 0, s>>>(a, run);
  return cudaGetLastError();
}

template <typename E, typename H, int kV>
cudaError_t by_width(const CacheCopyArgs& a, bool write, cudaStream_t s) {
  const int lanes = a.c.d / kV;
  if (lanes <= 1) return launch_t<E, H, kV, 1>(a, write, s);
  if (lanes <= 2) return launch_t<E, H, kV, 2>(a, write, s);
  if (lanes <= 4) return launch_t<E, H, kV, 4>(a, write, s);
  if (lanes <= 8) return launch_t<E, H, kV, 8>(a, write, s);
  if (lanes <= 16) return launch_t<E, H, kV, 16>(a, write, s);
  return launch_t<E, H, kV, 32>(a, write, s);
}

template <typename E, typename H>
cudaError_t by_vector(const CacheCopyArgs& a, bool write, cudaStream_t s) {
  return write && a.c.d % 16 == 0 ? by_width<E, H, 16>(a, write, s) : by_width<E, H, 8>(a, write, s);
}

cudaError_t dispatch(const CacheCopyArgs& a, ra_dtype dense, ra_dtype held, bool write,
                     cudaStream_t s) {
  if (dense == RA_BF16)
    return held == RA_E4M3 ? by_vector<__nv_bfloat16, __nv_fp8_e4m3>(a, write, s)
                           : by_vector<__nv_bfloat16, __nv_bfloat16>(a, write, s);
  return held == RA_E4M3 ? by_vector<float, __nv_fp8_e4m3>(a, write, s)
                         : by_vector<float, float>(a, write, s);
}

}  // namespace

cudaError_t launch_cache_write(const CacheCopyArgs& a, ra_dtype dense, ra_dtype held,
                               cudaStream_t s) {
  return dispatch(a, dense, held, true, s);
}

cudaError_t launch_cache_read(const CacheCopyArgs& a, ra_dtype dense, ra_dtype held,
                              cudaStream_t s) {
  return dispatch(a, dense, held, false, s);
}

}  // namespace ra
