// Attention of new tokens over the paged cache: the FFMA kernel (fp32
// inputs), the join of parts, and the choice of kernel.
//
// The FFMA kernel.  A unit is 16 query rows of one key head; 4 warps, each
// with 4 rows.  A tile of 32 keys is brought to shared memory as fp32 (8-bit
// rows multiplied by their scale); lane = key for the scores, lane = columns
// for P V, so the online softmax of a row stays inside its warp:
//   m' = max(m, max s),  l' = l e^(m-m') + sum p,  o' = o e^(m-m') + p V
// A key that a row does not see has p = 0 and is left out of the sum rather
// than multiplied, so what it holds does not matter.  Four CTAs share an SM and
// hide one another's loads; a CTA takes single tiles while there are few, since
// a tile's chain of look-up, load, scores and sum is what a short call waits
// for.

#include "ra_cache_attn.cuh"

namespace ra {
namespace {

constexpr int kRows = 16;
constexpr int kTile = 32;
constexpr int kThreads = 128;
constexpr int kColumns = RA_MAX_HEAD_DIM / 32;  // per lane
constexpr int kMaxSmem = (kRows * RA_MAX_HEAD_DIM + kTile * (2 * RA_MAX_HEAD_DIM + 4)) * 4;

template <typename E>
__device__ __forceinline__ float to_float(E x) {
  return static_cast<float>(x);
}
__device__ __forceinline__ void store_out(float* p, float x) { *p = x; }

__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                            *reinterpret_cast<const uint32_t*>(&hi));
}

template <typename E, typename H>
__global__ void __launch_bounds__(kThreads, 4)
    cache_attn_ffma_kernel(const __grid_constant__ CacheAttnArgs a,
                           const __grid_constant__ AttnPlan p) {
  constexpr bool k8 = sizeof(H) == 1;
  extern __shared__ float4 smem4[];
  __shared__ DivisionShared sh;
  __shared__ int64_t key_row[kTile];
  __shared__ float4 probs[4][kTile];  // of a warp's 4 rows, per key
  const PagedArgs& c = a.c;
  const int d = c.d, ld = d + 4;
  float* qs = reinterpret_cast<float*>(smem4);  // [kRows][d]
  float* ks = qs + kRows * d;                   // [kTile][ld]
  float* vs = ks + kTile * ld;                  // [kTile][d]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t rows = head_rows(a);

  allow_join();
  const int64_t run = division_start(c, p.div, blockIdx.x, sh);
  UnitWalk u;
  for (u.start(c, p.div, sh, run); !u.done(); u.next(c, p.div)) {
    const int head = u.unit / p.row_tiles;
    const int64_t r0 = static_cast<int64_t>(u.unit % p.row_tiles) * kRows;
    // q, out, lse row of row 0 of the unit
    const int64_t q0 = (static_cast<int64_t>(u.b) * c.heads + head) * rows + r0;
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * d; i += kThreads) {
      const int r = i / d;
      qs[i] = r0 + r < rows ? to_float(static_cast<const E*>(a.q)[q0 * d + i]) * a.scale_log2 : 0.f;
    }
    float m[4], l[4], o[4][kColumns];
    int t[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
      const int64_t row = r0 + 4 * warp + r;
      t[r] = row < rows ? static_cast<int>(row % c.T) : c.T;
#pragma unroll
      for (int x = 0; x < kColumns; ++x) o[r][x] = 0.f;
    }
    for (int64_t tile = u.first; tile < u.last; ++tile) {
      const int64_t pos0 = tile * kTile;
      __syncthreads();
      if (threadIdx.x < kTile) {
        const int64_t pos = pos0 + threadIdx.x;
        int64_t row = -1;
        if (pos < u.seq.keys()) row = cache_row(c, u.b, pos);
        key_row[threadIdx.x] = row < 0 ? -1 : row + (static_cast<int64_t>(head) << c.page_shift);
      }
      __syncthreads();
      for (int i0 = threadIdx.x; i0 < kTile * d / 8; i0 += 4 * kThreads) {
        // four pieces of 8 elements of K and of V are on their way together
        Packed<H, 8> x[4], y[4];
        uint32_t ek[4], ev[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int i = i0 + z * kThreads;
          const int key = i / (d / 8), e = (i % (d / 8)) * 8;
          const int64_t row = i < kTile * d / 8 ? key_row[key] : -1;
          x[z].zero();
          y[z].zero();
          ek[z] = ev[z] = 127;
          if (row >= 0) {
            x[z].load(static_cast<const H*>(c.k) + row * d + e);
            y[z].load(static_cast<const H*>(c.v) + row * d + e);
            if (k8) {
              ek[z] = c.ke[row];
              ev[z] = c.ve[row];
            }
          }
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int i = i0 + z * kThreads;
          if (i >= kTile * d / 8) break;
          const int key = i / (d / 8), e = (i % (d / 8)) * 8;
          float f[8];
          x[z].get(f);
          if (k8) {
            const float sk = exp_scale(ek[z]);
#pragma unroll
            for (int w = 0; w < 8; ++w) f[w] *= sk;
          }
          store8(ks + key * ld + e, f);
          y[z].get(f);
          if (k8) {
            const float sv = exp_scale(ev[z]);
#pragma unroll
            for (int w = 0; w < 8; ++w) f[w] *= sv;
          }
          store8(vs + key * d + e, f);
        }
      }
      __syncthreads();
      // scores of key `lane` for the warp's rows
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      for (int e = 0; e < d; e += 4) {
        const float4 kk = *reinterpret_cast<const float4*>(ks + lane * ld + e);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 qq = *reinterpret_cast<const float4*>(qs + (4 * warp + r) * d + e);
          s[r] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, s[r]))));
        }
      }
      const bool here = key_row[lane] >= 0;
      float pr4[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool seen = here && sees(a, u.seq, u.b, t[r], pos0 + lane);
        if (!seen) s[r] = -INFINITY;
        float mx = s[r];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        mx = fmaxf(mx, m[r]);
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float alpha = exp2f(m[r] - ref);  // 0 for an empty state
        const float pr = seen ? exp2f(s[r] - ref) : 0.f;
        float sum = pr;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l[r] = l[r] * alpha + sum;
        m[r] = mx;
        pr4[r] = pr;
#pragma unroll
        for (int x = 0; x < kColumns; ++x) o[r][x] *= alpha;
      }
      probs[warp][lane] = make_float4(pr4[0], pr4[1], pr4[2], pr4[3]);
      __syncwarp();
      if (r0 + 4 * warp < rows) {
#pragma unroll 4
        for (int key = 0; key < kTile; ++key) {
          const float4 pr = probs[warp][key];
#pragma unroll
          for (int x = 0; x < kColumns; ++x) {
            if (32 * x >= d) break;
            const int col = lane + 32 * x;
            const float vv = vs[key * d + (col < d ? col : 0)];
            o[0][x] = fmaf(pr.x, pr.x != 0.f ? vv : 0.f, o[0][x]);
            o[1][x] = fmaf(pr.y, pr.y != 0.f ? vv : 0.f, o[1][x]);
            o[2][x] = fmaf(pr.z, pr.z != 0.f ? vv : 0.f, o[2][x]);
            o[3][x] = fmaf(pr.w, pr.w != 0.f ? vv : 0.f, o[3][x]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = r0 + 4 * warp + r;
      if (row >= rows) continue;
      if (u.whole()) {
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
        E* dst = static_cast<E*>(a.out) + (q0 + 4 * warp + r) * d;
#pragma unroll
        for (int x = 0; x < kColumns; ++x)
          if (lane + 32 * x < d) store_out(dst + lane + 32 * x, o[r][x] * inv);
        if (lane == 0)
          a.lse[q0 + 4 * warp + r] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2F;
      } else {
        const int slot = u.slot(blockIdx.x);
        float* dst = slot_o(a, p, slot) + (4 * warp + r) * d;
#pragma unroll
        for (int x = 0; x < kColumns; ++x)
          if (lane + 32 * x < d) dst[lane + 32 * x] = o[r][x];
        if (lane == 0) {
          float* ml = slot_ml(a, p, slot) + (4 * warp + r) * 2;
          ml[0] = m[r];
          ml[1] = l[r];
        }
      }
    }
  }
}

// ------------------------------------------------------------------- join
// A query row whose unit was shared is joined by `kSplit` warps: its parts lie
// in the slots of consecutive CTAs, a warp takes every kSplit-th, four at a
// time (the loads of four parts are in flight together), and the warps' sums
// are added in order.  blockIdx.y is the sequence; the units' places follow
// from the lengths, as in the walk.  Every slot of a shared unit has been
// written, an empty part with l = 0 and o = 0.
constexpr int kJoinWarps = 8;

template <typename E, int kSplit>
__global__ void __launch_bounds__(kJoinWarps * 32)
    cache_attn_join_kernel(const __grid_constant__ CacheAttnArgs a,
                           const __grid_constant__ AttnPlan p) {
  __shared__ DivisionShared sh;
  __shared__ int64_t before;
  __shared__ float4 sums[kJoinWarps][2][32];
  __shared__ float sum_l[kJoinWarps];
  const PagedArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sub = warp % kSplit;
  const int64_t rows = head_rows(a);
  const int64_t seq_rows = rows * c.heads;
  for (int b = blockIdx.y; b < c.B; b += gridDim.y) {
    // tiles (of one unit) of the sequences before b, and of all
    int64_t ahead, total;
    if (c.B <= 32) {
      const int64_t upto = warp_scan(lane < c.B ? seq_tiles(c, p.div, lane) : 0);
      ahead = b > 0 ? __shfl_sync(0xffffffffu, upto, b - 1) : 0;
      total = __shfl_sync(0xffffffffu, upto, 31);
    } else {
      __syncthreads();
      int64_t mine = 0, all = 0;
      for (int i = threadIdx.x; i < c.B; i += blockDim.x) {
        const int64_t t = seq_tiles(c, p.div, i);
        all += t;
        if (i < b) mine += t;
      }
      const int64_t x = block_scan(mine, sh);
      if (threadIdx.x == blockDim.x - 1) before = x;
      __syncthreads();
      block_scan(all, sh);
      __syncthreads();
      ahead = before;
      total = sh.total;
    }
    if (c.count && blockIdx.x == 0 && threadIdx.x == 0 && c.lens[b] >= 0 && c.count[b] > c.T)
      flag_page(c.status);
    const int64_t per = run_length(p.div, total * p.div.units);
    const int64_t tiles = seq_tiles(c, p.div, b);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kJoinWarps / kSplit) + warp / kSplit;
    int c0 = 0, c1 = 0, local = 0;
    if (row < seq_rows) {
      const int64_t in_head = row % rows;
      const int unit = static_cast<int>(row / rows) * p.row_tiles +
                       static_cast<int>(in_head / p.rows);
      local = static_cast<int>(in_head % p.rows);
      const int64_t u0 = ahead * p.div.units + unit * tiles;
      c0 = static_cast<int>(u0 / per);
      c1 = static_cast<int>((u0 + tiles - 1) / per);
    }
    const bool shared = c1 > c0;
    wait_for_parts();
    float ms = -INFINITY, l = 0.f;
    float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (shared) {
      for (int i = c0 + lane; i <= c1; i += 32)
        ms = fmaxf(ms, slot_ml(a, p, 2 * i + (i == c0 ? 1 : 0))[2 * local]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, off));
      const float ref = ms == -INFINITY ? 0.f : ms;
      for (int i = c0 + sub; i <= c1; i += 4 * kSplit) {
        float2 ml[4];
        float4 y[4][2];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int at = i + z * kSplit;
          const bool real = at <= c1;
          const int slot = real ? 2 * at + (at == c0 ? 1 : 0) : 0;
          ml[z] = real ? *reinterpret_cast<const float2*>(slot_ml(a, p, slot) + 2 * local)
                       : make_float2(-INFINITY, 0.f);
          const float4* src =
              reinterpret_cast<const float4*>(slot_o(a, p, slot) + static_cast<int64_t>(local) * c.d);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            y[z][h] = real && 4 * (lane + 32 * h) < c.d ? src[lane + 32 * h]
                                                         : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float w = ml[z].y == 0.f ? 0.f : exp2f(ml[z].x - ref);
          l = fmaf(w, ml[z].y, l);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            o[h].x = fmaf(w, y[z][h].x, o[h].x);
            o[h].y = fmaf(w, y[z][h].y, o[h].y);
            o[h].z = fmaf(w, y[z][h].z, o[h].z);
            o[h].w = fmaf(w, y[z][h].w, o[h].w);
          }
        }
      }
    }
    if (kSplit > 1) {
      sums[warp][0][lane] = o[0];
      sums[warp][1][lane] = o[1];
      if (lane == 0) sum_l[warp] = l;
      __syncthreads();
      if (sub == 0) {
        for (int z = 1; z < kSplit; ++z) {
          l += sum_l[warp + z];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 y = sums[warp + z][h][lane];
            o[h].x += y.x;
            o[h].y += y.y;
            o[h].z += y.z;
            o[h].w += y.w;
          }
        }
      }
    }
    if (shared && sub == 0) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t at = static_cast<int64_t>(b) * seq_rows + row;
      E* dst = static_cast<E*>(a.out) + at * c.d;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = 4 * (lane + 32 * h);
        if (col < c.d) store4(dst + col, make_float4(o[h].x * inv, o[h].y * inv, o[h].z * inv, o[h].w * inv));
      }
      if (lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (ms + log2f(l)) * kLn2F;
    }
  }
}

AttnPlan ffma_plan(const CacheAttnArgs& a) {
  AttnPlan p;
  p.rows = kRows;
  p.row_tiles = static_cast<int>((head_rows(a) + kRows - 1) / kRows);
  p.div.units = a.c.heads * p.row_tiles;
  p.div.tile = kTile;
  p.div.ctas = kFfmaCtas;
  p.div.min_run = 1;
  return p;
}

template <typename E, int kSplit>
cudaError_t join_t(const CacheAttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  const int64_t seq_rows = head_rows(a) * a.c.heads;
  constexpr int kRowsPerBlock = kJoinWarps / kSplit;
  const dim3 grid(static_cast<unsigned>((seq_rows + kRowsPerBlock - 1) / kRowsPerBlock),
                  static_cast<unsigned>(a.c.B < 65535 ? a.c.B : 65535));
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<E, kSplit>, a, p);
}

template <typename E, typename H>
cudaError_t launch_ffma(const CacheAttnArgs& a, cudaStream_t s) {
  const AttnPlan p = ffma_plan(a);
  const int smem = (kRows * a.c.d + kTile * (2 * a.c.d + 4)) * 4;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(cache_attn_ffma_kernel<E, H>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cache_attn_ffma_kernel<E, H><<<p.div.ctas, kThreads, smem, s>>>(a, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_cache_attn_join(a, p, sizeof(E) == 2, s);
}

}  // namespace

cudaError_t launch_cache_attn_join(const CacheAttnArgs& a, const AttnPlan& p, bool bf16,
                                   cudaStream_t s) {
  // A unit is shared by about ctas / units CTAs.  A warp takes the parts of a
  // row four at a time; with more than two such rounds several share the row.
  const int64_t units = static_cast<int64_t>(a.c.B) * p.div.units;
  if (p.div.ctas > 48 * units) return bf16 ? join_t<__nv_bfloat16, 8>(a, p, s) : join_t<float, 8>(a, p, s);
  if (p.div.ctas > 8 * units) return bf16 ? join_t<__nv_bfloat16, 2>(a, p, s) : join_t<float, 2>(a, p, s);
  return bf16 ? join_t<__nv_bfloat16, 1>(a, p, s) : join_t<float, 1>(a, p, s);
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a, ra_dtype dense, ra_dtype held,
                                   cudaStream_t s) {
  if (dense == RA_F32)
    return held == RA_E4M3 ? launch_ffma<float, __nv_fp8_e4m3>(a, s) : launch_ffma<float, float>(a, s);
  // The decode kernel reads a key head once per 16 query rows, the tree kernel
  // once per 256.  Up to 16 rows the former is ahead throughout.  With 17 to 32
  // rows it still is over 8-bit caches, which the tree kernel has to widen
  // (16 sequences of 16384, 8 heads, 32 rows: 190 against 242 us; bf16: 331
  // against 182).
  const int most = held == RA_E4M3 ? 2 * kDecodeRows : kDecodeRows;
  if (head_rows(a) > most) return launch_cache_tree(a, held == RA_E4M3, s);
  return launch_cache_decode(a, held == RA_E4M3, s);
}

int64_t cache_attention_workspace_bytes(int32_t B, int32_t Hq, int32_t heads, int32_t T,
                                        int32_t d) {
  // The largest of the kernels that may serve these sizes (the types are not
  // known here): parts of 2 slots per CTA.
  (void)B;
  const int64_t rows = static_cast<int64_t>(Hq / heads) * T;
  int64_t most = kFfmaCtas * kRows;
  if (rows > kDecodeRows) most = kTreeCtas * (rows > 128 ? 256 : 128);
  if (most < kFfmaCtas * kRows) most = kFfmaCtas * kRows;
  return 2 * most * (d + 2) * 4;
}

}  // namespace ra
