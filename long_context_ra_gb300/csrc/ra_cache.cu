// Writing new tokens into a paged K/V cache (quantising them for an 8-bit
// one) and reading positions back.
//
// Bound by memory: every element crosses once.  A row of d elements belongs
// to d / 8 lanes (padded to a power of two for the row's maximum), 8
// elements a lane.  A group of lanes takes one token, finds its page once and
// walks over a run of the 2 x heads rows of K and V, the loads of kAhead rows
// in flight together; neighbouring groups hold neighbouring tokens, whose
// rows lie next to each other in a page.

#include "ra_paged.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;

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

template <typename E, typename H, int kLanes>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheCopyArgs a,
                                                               int run) {
  constexpr bool k8 = !Same<E, H>::value;
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
  const bool live = base >= 0 && 8 * l < c.d;
  const int r_end = min(2 * c.heads, static_cast<int>(blockIdx.y + 1) * run);
  for (int r0 = blockIdx.y * run; r0 < r_end; r0 += kAhead) {
    float x[kAhead][8];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = r0 + j;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
      if (r < r_end && live) {
        const bool v = r >= c.heads;
        const Strides& st = v ? a.vs : a.ks;
        const int h = v ? r - c.heads : r;
        load8(static_cast<const E*>(v ? a.v : a.k) + b * st.b + h * st.h + t * st.n + 8 * l, x[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = r0 + j;
      if (r >= r_end) break;
      const bool v = r >= c.heads;
      const int h = v ? r - c.heads : r;
      const int64_t row = base + (static_cast<int64_t>(h) << c.page_shift);
      if (k8) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = fabsf(x[j][i]);
          m = y < INFINITY ? fmaxf(m, y) : m;  // finite elements only
        }
        const uint32_t e = row_exponent(row_max<kLanes>(m));
        const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= inv;
        if (live) {
          uint8_t* p = static_cast<uint8_t*>(v ? c.v : c.k) + row * c.d + 8 * l;
          *reinterpret_cast<uint2*>(p) = make_uint2(pack_e4m3x4(x[j]), pack_e4m3x4(x[j] + 4));
          if (l == 0) (v ? c.ve : c.ke)[row] = static_cast<uint8_t>(e);
        }
      } else if (live) {
        store8(static_cast<E*>(v ? c.v : c.k) + row * c.d + 8 * l, x[j]);
      }
    }
  }
}

template <typename E, typename H, int kLanes>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheCopyArgs a,
                                                              int run) {
  constexpr bool k8 = !Same<E, H>::value;
  const PagedArgs& c = a.c;
  const int l = threadIdx.x % kLanes;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (token >= c.B * a.n || 8 * l >= c.d) return;
  const int b = static_cast<int>(token / a.n);
  const int64_t n = token % a.n;
  const int64_t base = a.first + n < c.lens[b] ? cache_row(c, b, a.first + n) : -1;
  const int r_end = min(2 * c.heads, static_cast<int>(blockIdx.y + 1) * run);
  for (int r0 = blockIdx.y * run; r0 < r_end; r0 += kAhead) {
    float x[kAhead][8];
    uint32_t e[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = r0 + j;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
      e[j] = 127;
      if (r < r_end && base >= 0) {
        const bool v = r >= c.heads;
        const int64_t row = base + (static_cast<int64_t>(v ? r - c.heads : r) << c.page_shift);
        load8(static_cast<const H*>(v ? c.v : c.k) + row * c.d + 8 * l, x[j]);
        if (k8) e[j] = (v ? c.ve : c.ke)[row];
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = r0 + j;
      if (r >= r_end) break;
      const bool v = r >= c.heads;
      const int h = v ? r - c.heads : r;
      if (k8) {
        const float sc = exp_scale(e[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= sc;
      }
      E* p = static_cast<E*>(v ? a.v : a.k) + ((static_cast<int64_t>(b) * c.heads + h) * a.n + n) * c.d;
      store8(p + 8 * l, x[j]);
    }
  }
}

// Rows per run: all 2 x heads of a token while that fills the SMs four
// times over, else fewer.
int rows_per_run(int64_t tiles, int rows) {
  const int64_t want = static_cast<int64_t>(device_sm_count()) * 4;
  int64_t runs = (want + tiles - 1) / tiles;
  if (runs > rows) runs = rows;
  return static_cast<int>((rows + runs - 1) / runs);
}

template <typename E, typename H, int kLanes>
cudaError_t launch_t(const CacheCopyArgs& a, bool write, cudaStream_t s) {
  const int64_t tokens = a.c.B * (write ? static_cast<int64_t>(a.c.T) : a.n);
  constexpr int kGroups = kThreads / kLanes;
  const int64_t tiles = (tokens + kGroups - 1) / kGroups;
  const int rows = 2 * a.c.heads;
  const int run = rows_per_run(tiles, rows);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((rows + run - 1) / run));
  if (write)
    cache_write_kernel<E, H, kLanes><<<grid, kThreads, 0, s>>>(a, run);
  else
    cache_read_kernel<E, H, kLanes><<<grid, kThreads, 0, s>>>(a, run);
  return cudaGetLastError();
}

template <typename E, typename H>
cudaError_t by_width(const CacheCopyArgs& a, bool write, cudaStream_t s) {
  const int d = a.c.d;
  if (d <= 16) return launch_t<E, H, 2>(a, write, s);
  if (d <= 32) return launch_t<E, H, 4>(a, write, s);
  if (d <= 64) return launch_t<E, H, 8>(a, write, s);
  if (d <= 128) return launch_t<E, H, 16>(a, write, s);
  return launch_t<E, H, 32>(a, write, s);
}

cudaError_t dispatch(const CacheCopyArgs& a, ra_dtype dense, ra_dtype held, bool write,
                     cudaStream_t s) {
  if (dense == RA_BF16)
    return held == RA_E4M3 ? by_width<__nv_bfloat16, __nv_fp8_e4m3>(a, write, s)
                           : by_width<__nv_bfloat16, __nv_bfloat16>(a, write, s);
  return held == RA_E4M3 ? by_width<float, __nv_fp8_e4m3>(a, write, s)
                         : by_width<float, float>(a, write, s);
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
