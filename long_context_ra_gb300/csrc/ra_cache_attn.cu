// Attention of new tokens over the paged cache: the FFMA kernel (fp32
// inputs), the join of parts, and the choice of kernel.
//
// The FFMA kernel.  A tile of keys is brought to shared memory as fp32 (8-bit
// rows multiplied by their scale).  A warp has kRW query rows and 32 kKL keys
// of the tile: lane = key for the scores, lane = columns for P V, so the
// online softmax of a row stays inside its warp:
//   m' = max(m, max s),  l' = l e^(m-m') + sum p,  o' = o e^(m-m') + p V
// As in the other kernels m moves only when a score passes it by 2^8, which a
// vote tells, and l is summed over the lanes at the end.  kRG warps take the
// rows, kKG the keys of a tile (their states are joined at the end of a unit),
// so that four rows keep four warps busy as well as 16 do.
//
// Few rows wait for the chain of look-up, load, scores and sum of each tile;
// three or more CTAs share an SM and hide one another's, the page look-up runs
// a tile ahead, and a CTA takes single tiles while there are few.  Many rows
// are bound by instructions: both products run on pairs (fma.rn.f32x2), of
// neighbouring elements for the scores and of neighbouring columns for P V,
// whose probabilities are kept twice side by side; 8 rows x 2 keys a lane are
// 32 paired FFMA for 10 reads of 16 bytes.  Measured: 2 sequences of 4096, 3 key
// heads of 80, 6 rows each 19 us a call (70 with one warp per row and a tile at
// a time); 256 rows over 4096 keys of 128: 17 TFLOP/s.
//
// A key that a row does not see has p = 0.  In tiles with drafts or the end that
// hold a value that is not finite it is left out of the sum rather than
// multiplied, so what it holds does not matter; -0 in place of p tells it from a
// key that is seen and whose p is 0.  (Leaving keys out costs a branch per key and
// row: 651 rows of 34 sequences of 98 keys 886 us, not 674.)

#include "ra_cache_attn.cuh"
#include "sm103_ptx.cuh"

namespace ra {
namespace {

using namespace ptx;

constexpr int kFfmaSmem = 192 * 1024;  // dynamic, beside 33 KB of static
constexpr float kSlack = 8.f;

__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                            *reinterpret_cast<const uint32_t*>(&hi));
}

// NC: pairs of columns of a head per lane, 2 (d <= 128) or 4.
template <int RW, int KL, int RG, int KG, int NC>
struct Ffma {
  static constexpr int kRW = RW, kKL = KL, kRG = RG, kKG = KG, kPairs = NC;
  static constexpr int kCtas = 32 * RG * KG > 128 ? (NC == 2 ? 2 : 1) : 4;  // per SM, by registers
  static constexpr int kWarps = RG * KG;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = RG * RW;
  static constexpr int kWarpKeys = 32 * KL;
  static constexpr int kTile = KG * kWarpKeys;
  // queries, K (pitch d + 4), V; the joined states take the place of K and V
  static int smem(int d) { return (kRows * d + kTile * (2 * d + 4)) * 4; }
};

template <typename H, typename F>
__global__ void __launch_bounds__(F::kThreads, F::kCtas)
    cache_attn_ffma_kernel(const __grid_constant__ CacheAttnArgs a,
                           const __grid_constant__ AttnPlan p) {
  constexpr bool k8 = sizeof(H) == 1;
  constexpr int kRW = F::kRW, kKL = F::kKL, kTile = F::kTile, kPairs = F::kPairs;
  extern __shared__ float4 smem4[];
  __shared__ DivisionShared sh;
  __shared__ int64_t key_row[2][kTile];
  __shared__ float4 probs[F::kWarps][F::kWarpKeys][kRW / 2];  // (p, p, p', p') of two rows
  __shared__ float states[F::kWarps][kRW][2];
  const PagedArgs& c = a.c;
  const int d = c.d, ld = d + 4;
  float* qs = reinterpret_cast<float*>(smem4);  // [kRows][d]
  float* ks = qs + F::kRows * d;                // [kTile][ld]
  float* vs = ks + kTile * ld;                  // [kTile][d]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rg = warp % F::kRG, kg = warp / F::kRG;
  const int64_t rows = head_rows(a);

  allow_join();
  const int64_t run = division_start(c, p.div, blockIdx.x, sh);
  UnitWalk u;
  for (u.start(c, p.div, sh, run); !u.done(); u.next(c, p.div)) {
    const int head = u.unit / p.row_tiles;
    const int64_t r0 = static_cast<int64_t>(u.unit % p.row_tiles) * F::kRows;
    // q, out, lse row of row 0 of the unit
    const int64_t q0 = (static_cast<int64_t>(u.b) * c.heads + head) * rows + r0;
    const int64_t keys = u.seq.keys(), context = u.seq.len;
    auto look_up = [&](int64_t tile) {
      if (threadIdx.x < kTile && tile < u.last) {
        const int64_t pos = tile * kTile + threadIdx.x;
        const int64_t row = pos < keys ? cache_row(c, u.b, pos) : -1;
        key_row[tile & 1][threadIdx.x] =
            row < 0 ? -1 : row + (static_cast<int64_t>(head) << c.page_shift);
      }
    };
    __syncthreads();
    look_up(u.first);
    const float* q = static_cast<const float*>(a.q) + q0 * d;
    for (int i = threadIdx.x * 4; i < F::kRows * d; i += F::kThreads * 4) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r0 + i / d < rows) x = *reinterpret_cast<const float4*>(q + i);
      const float t = a.scale_log2;
      *reinterpret_cast<float4*>(qs + i) = make_float4(x.x * t, x.y * t, x.z * t, x.w * t);
    }
    float m[kRW], l[kRW];
    uint64_t o[kRW][kPairs];  // columns 2 lane, 2 lane + 1 of every 64
    int t[kRW];
#pragma unroll
    for (int r = 0; r < kRW; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
      const int64_t row = r0 + rg * kRW + r;
      t[r] = row < rows ? static_cast<int>(row % c.T) : c.T;
#pragma unroll
      for (int x = 0; x < kPairs; ++x) o[r][x] = 0ull;
    }
    for (int64_t tile = u.first; tile < u.last; ++tile) {
      const int64_t* at = key_row[tile & 1];
      __syncthreads();
      look_up(tile + 1);
      const bool border = tile * kTile + kTile > context;
      bool bad = false;  // a value that is not finite in a tile that not every row sees
      for (int i0 = threadIdx.x; i0 < kTile * d / 8; i0 += 4 * F::kThreads) {
        // four pieces of 8 elements of K and of V are on their way together
        Packed<H, 8> x[4], y[4];
        uint32_t ek[4], ev[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int i = i0 + z * F::kThreads;
          const int64_t row = i < kTile * d / 8 ? at[i / (d / 8)] : -1;
          x[z].zero();
          y[z].zero();
          ek[z] = ev[z] = 127;
          if (row >= 0) {
            const int e = (i % (d / 8)) * 8;
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
          const int i = i0 + z * F::kThreads;
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
          if (border) {
#pragma unroll
            for (int w = 0; w < 8; ++w) bad = bad || !(fabsf(f[w]) < INFINITY);
          }
          store8(vs + key * d + e, f);
        }
      }
      const bool clean = !__syncthreads_or(bad);
      if (r0 + rg * kRW >= rows) continue;  // no row of this warp's
      // ---- scores of keys lane, lane + 32 of the warp's part of the tile
      const float* kw = ks + (kg * F::kWarpKeys + lane) * ld;
      const float* qw = qs + rg * kRW * d;
      uint64_t s2[kRW][kKL];
#pragma unroll
      for (int r = 0; r < kRW; ++r)
#pragma unroll
        for (int z = 0; z < kKL; ++z) s2[r][z] = 0ull;
#pragma unroll 2
      for (int e = 0; e < d; e += 4) {
        ulonglong2 kk[kKL];
#pragma unroll
        for (int z = 0; z < kKL; ++z) kk[z] = *reinterpret_cast<const ulonglong2*>(kw + 32 * z * ld + e);
#pragma unroll
        for (int r = 0; r < kRW; ++r) {
          const ulonglong2 qq = *reinterpret_cast<const ulonglong2*>(qw + r * d + e);
#pragma unroll
          for (int z = 0; z < kKL; ++z)
            s2[r][z] = fma_f32x2(qq.x, kk[z].x, fma_f32x2(qq.y, kk[z].y, s2[r][z]));
        }
      }
      float s[kRW][kKL];
#pragma unroll
      for (int r = 0; r < kRW; ++r)
#pragma unroll
        for (int z = 0; z < kKL; ++z) {
          float lo, hi;
          unpack_f32x2(s2[r][z], lo, hi);
          s[r][z] = lo + hi;
        }
      const int64_t pos0 = tile * kTile + kg * F::kWarpKeys;
      bool whole_tile = pos0 + F::kWarpKeys <= context;  // every row sees every key
#pragma unroll
      for (int z = 0; z < kKL; ++z) whole_tile = whole_tile && at[kg * F::kWarpKeys + lane + 32 * z] >= 0;
      whole_tile = __all_sync(0xffffffffu, whole_tile);
      if (!whole_tile) {
#pragma unroll
        for (int z = 0; z < kKL; ++z) {
          const int64_t pos = pos0 + lane + 32 * z;
          const bool here = at[kg * F::kWarpKeys + lane + 32 * z] >= 0;
#pragma unroll
          for (int r = 0; r < kRW; ++r)
            if (!here || !sees(a, u.seq, u.b, t[r], pos)) s[r][z] = -INFINITY;
        }
      }
      // ---- reference, probabilities
      bool pass = false;
#pragma unroll
      for (int r = 0; r < kRW; ++r)
#pragma unroll
        for (int z = 0; z < kKL; ++z) pass = pass || s[r][z] > m[r] + kSlack;
      if (__any_sync(0xffffffffu, pass)) {
#pragma unroll
        for (int r = 0; r < kRW; ++r) {
          float x = m[r];
#pragma unroll
          for (int z = 0; z < kKL; ++z) x = fmaxf(x, s[r][z]);
#pragma unroll
          for (int w = 16; w > 0; w >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
          const float alpha = m[r] == x ? 1.f : exp2f(m[r] - x);
          m[r] = x;
          l[r] *= alpha;
#pragma unroll
          for (int z = 0; z < kPairs; ++z) o[r][z] = mul_f32x2(o[r][z], pack_f32x2(alpha, alpha));
        }
      }
#pragma unroll
      for (int z = 0; z < kKL; ++z) {
#pragma unroll
        for (int r = 0; r < kRW; r += 2) {
          const float p0 = exp2f(s[r][z] - (m[r] == -INFINITY ? 0.f : m[r]));
          const float p1 = exp2f(s[r + 1][z] - (m[r + 1] == -INFINITY ? 0.f : m[r + 1]));
          l[r] += p0;
          l[r + 1] += p1;
          probs[warp][lane + 32 * z][r / 2] = make_float4(p0, p0, p1, p1);
        }
      }
      if (!whole_tile && !clean) {  // -0 for keys that are not seen: a seen one's p may be 0
#pragma unroll
        for (int z = 0; z < kKL; ++z) {
          const int64_t pos = pos0 + lane + 32 * z;
          const bool here = at[kg * F::kWarpKeys + lane + 32 * z] >= 0;
          float2* pr = reinterpret_cast<float2*>(probs[warp][lane + 32 * z]);
#pragma unroll
          for (int r = 0; r < kRW; ++r)
            if (!here || !sees(a, u.seq, u.b, t[r], pos)) pr[r] = make_float2(-0.f, -0.f);
        }
      }
      __syncwarp();
      // ---- values
      const float* vw = vs + kg * F::kWarpKeys * d;
      int col[kPairs];
#pragma unroll
      for (int x = 0; x < kPairs; ++x) col[x] = 2 * lane + 64 * x < d ? 2 * lane + 64 * x : 0;
#pragma unroll 2
      for (int key = 0; key < F::kWarpKeys; ++key, vw += d) {
        ulonglong2 pr[kRW / 2];
#pragma unroll
        for (int r = 0; r < kRW / 2; ++r) pr[r] = *reinterpret_cast<const ulonglong2*>(&probs[warp][key][r]);
        uint64_t vv[kPairs];
#pragma unroll
        for (int x = 0; x < kPairs; ++x)
          if (64 * x < d) vv[x] = *reinterpret_cast<const uint64_t*>(vw + col[x]);
        if (whole_tile || clean) {
#pragma unroll
          for (int x = 0; x < kPairs; ++x)
            if (64 * x < d) {
#pragma unroll
              for (int r = 0; r < kRW; r += 2) {
                o[r][x] = fma_f32x2(pr[r / 2].x, vv[x], o[r][x]);
                o[r + 1][x] = fma_f32x2(pr[r / 2].y, vv[x], o[r + 1][x]);
              }
            }
        } else {
#pragma unroll
          for (int r = 0; r < kRW; r += 2) {
            // the same for every lane: whether a row sees this key
            constexpr uint64_t unseen = 0x8000000080000000ull;
            const bool s0 = pr[r / 2].x != unseen, s1 = pr[r / 2].y != unseen;
#pragma unroll
            for (int x = 0; x < kPairs; ++x)
              if (64 * x < d) {
                if (s0) o[r][x] = fma_f32x2(pr[r / 2].x, vv[x], o[r][x]);
                if (s1) o[r + 1][x] = fma_f32x2(pr[r / 2].y, vv[x], o[r + 1][x]);
              }
          }
        }
      }
      __syncwarp();
    }
    // ---- join the key groups' states, then out, or this CTA's part
#pragma unroll
    for (int r = 0; r < kRW; ++r)
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
    float* parts = ks;  // [kKG - 1][kRows][d]
    if (F::kKG > 1) {
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRW; ++r) {
        if (lane == 0) {
          states[warp][r][0] = m[r];
          states[warp][r][1] = l[r];
        }
        if (kg > 0) {
#pragma unroll
          for (int x = 0; x < kPairs; ++x)
            if (2 * lane + 64 * x < d)
              *reinterpret_cast<uint64_t*>(
                  parts + ((kg - 1) * F::kRows + rg * kRW + r) * d + 2 * lane + 64 * x) = o[r][x];
        }
      }
      __syncthreads();
    }
    if (kg > 0) continue;
#pragma unroll
    for (int r = 0; r < kRW; ++r) {
      const int local = rg * kRW + r;
      if (r0 + local >= rows) continue;
      if (F::kKG > 1) {
        float ms = m[r];
#pragma unroll
        for (int g = 1; g < F::kKG; ++g) ms = fmaxf(ms, states[g * F::kRG + rg][r][0]);
        const float ref = ms == -INFINITY ? 0.f : ms;
        // A weight of 0 multiplies too: o may be NaN, and is 0 without a seen key.
        const float f0 = l[r] == 0.f ? 0.f : exp2f(m[r] - ref);
        float ls = f0 * l[r];
#pragma unroll
        for (int x = 0; x < kPairs; ++x) o[r][x] = mul_f32x2(o[r][x], pack_f32x2(f0, f0));
#pragma unroll
        for (int g = 1; g < F::kKG; ++g) {
          const float lg = states[g * F::kRG + rg][r][1];
          const float f = lg == 0.f ? 0.f : exp2f(states[g * F::kRG + rg][r][0] - ref);
          ls += f * lg;
#pragma unroll
          for (int x = 0; x < kPairs; ++x)
            if (2 * lane + 64 * x < d)
              o[r][x] = fma_f32x2(pack_f32x2(f, f),
                                  *reinterpret_cast<const uint64_t*>(
                                      parts + ((g - 1) * F::kRows + local) * d + 2 * lane + 64 * x),
                                  o[r][x]);
        }
        m[r] = ms;
        l[r] = ls;
      }
      const bool dead = t[r] >= u.seq.cnt;  // no query: an empty state
      if (dead) {
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
      const bool whole = u.whole();
      const float f = l[r] == 0.f ? 0.f : whole ? 1.f / l[r] : 1.f;
      const int slot = u.slot(blockIdx.x);
      float* dst = whole ? static_cast<float*>(a.out) + (q0 + local) * d
                         : slot_o(a, p, slot) + static_cast<int64_t>(local) * d;
#pragma unroll
      for (int x = 0; x < kPairs; ++x)
        if (2 * lane + 64 * x < d)
          *reinterpret_cast<uint64_t*>(dst + 2 * lane + 64 * x) =
              dead ? 0ull : mul_f32x2(o[r][x], pack_f32x2(f, f));
      if (lane == 0) {
        if (whole) {
          a.lse[q0 + local] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2F;
        } else {
          float* ml = slot_ml(a, p, slot) + 2 * local;
          ml[0] = m[r];
          ml[1] = l[r];
        }
      }
    }
  }
}

// ------------------------------------------------------------------- join
// Only units that the border between two CTAs' runs cuts have parts.
// blockIdx.y is a unit, or, where there are fewer of those, such a border: the
// first one inside a unit stands for it.  The blocks of others have nothing to
// join, but wait as well: what follows the join on the stream may only begin
// when the kernel before it has ended.
// blockIdx.x is a group of the unit's rows.
// A row is joined by kSplit warps: its parts lie in the slots of consecutive
// CTAs, a warp takes every kSplit-th, four at a time (the loads of four parts
// are in flight together), and the warps' sums are added in order.  Every slot
// of a shared unit has been written, an empty part with l = 0 and o = 0.
// A lane holds kCols times 4 columns: 1 up to d = 128, which keeps the block at
// 64 registers a thread, four blocks on an SM (8 sequences of 32 tokens: 97.7
// -> 96.2 us; eight parts in flight take 98 registers: 100.3 us).
constexpr int kJoinWarps = 8;

// A unit that has parts: false where the block has none to join.
struct Shared {
  int64_t q0;   // row of the unit's first row in q, out, lse
  int some;     // rows of the unit
  int c0, c1;   // the CTAs that shared it
};

__device__ bool shared_unit(const CacheAttnArgs& a, const AttnPlan& p, bool by_unit, DivisionShared& sh,
                            Shared& j) {
  const PagedArgs& c = a.c;
  int b, unit;
  if (by_unit) {
    b = blockIdx.y / p.div.units;
    unit = blockIdx.y % p.div.units;
    int64_t ahead, total;
    division_before(c, p.div, b, sh, ahead, total);
    const int64_t tiles = seq_tiles(c, p.div, b), run = run_length(p.div, total * p.div.units);
    const int64_t u0 = ahead * p.div.units + unit * tiles;
    j.c0 = static_cast<int>(u0 / run);
    j.c1 = static_cast<int>((u0 + tiles - 1) / run);
    if (j.c0 == j.c1) return false;
  } else {
    const int border = blockIdx.y + 1;
    if (division_start(c, p.div, border, sh) == 0) return false;
    b = sh.b;
    const int64_t tiles = tiles_of(sh.seq, p.div);
    unit = static_cast<int>(sh.off / tiles);
    const int64_t inside = sh.off - unit * tiles;  // tiles of the unit before the border
    // a unit begins here, or was cut before
    if (inside == 0 || inside > sh.run) return false;
    j.c0 = border - 1;
    j.c1 = static_cast<int>((border * sh.run - inside + tiles - 1) / sh.run);
  }
  const int64_t rows = head_rows(a);
  const int64_t r0 = static_cast<int64_t>(unit % p.row_tiles) * p.rows;
  j.q0 = (static_cast<int64_t>(b) * c.heads + unit / p.row_tiles) * rows + r0;
  j.some = static_cast<int>(min(rows - r0, static_cast<int64_t>(p.rows)));
  return true;
}

template <typename E, int kSplit, int kCols>
__global__ void __launch_bounds__(kJoinWarps * 32)
    cache_attn_join_kernel(const __grid_constant__ CacheAttnArgs a,
                           const __grid_constant__ AttnPlan p, int block_rows, bool by_unit) {
  __shared__ DivisionShared sh;
  __shared__ float4 sums[kJoinWarps][kCols][32];
  __shared__ float sum_l[kJoinWarps];
  constexpr int kStep = kJoinWarps / kSplit;  // rows at a time
  constexpr int kParts = 4;
  const PagedArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sub = warp % kSplit;
  Shared j;
  if (!shared_unit(a, p, by_unit, sh, j)) return wait_for_parts();
  const int64_t q0 = j.q0;
  const int some = j.some, c0 = j.c0, c1 = j.c1;
  // rows of all slots: fewer than 2^17, of d floats each
  const float2* all_ml = reinterpret_cast<const float2*>(slot_ml(a, p, 0));
  const float4* all_o = reinterpret_cast<const float4*>(slot_o(a, p, 0));
  const uint32_t quads = c.d / 4;
  wait_for_parts();
  const int begin = blockIdx.x * block_rows, end = min(some, begin + block_rows);
  for (int first = begin; first < end; first += kStep) {
    const int local = first + warp / kSplit;
    const bool shared = local < end;
    float ms = -INFINITY, l = 0.f;
    float4 o[kCols];
#pragma unroll
    for (int h = 0; h < kCols; ++h) o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (shared) {
      // the loads of a round's parts, which need no weight yet
      float2 ml[kParts];
      float4 y[kParts][kCols];
      auto fetch = [&](int i) {
#pragma unroll
        for (int z = 0; z < kParts; ++z) {
          const int at = i + z * kSplit;
          const bool real = at <= c1;
          const uint32_t row = (2u * at + (at == c0 ? 1u : 0u)) * p.rows + local;
          ml[z] = real ? all_ml[row] : make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int h = 0; h < kCols; ++h)
            y[z][h] = real && lane + 32 * h < quads ? all_o[row * quads + lane + 32 * h]
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      };
      fetch(c0 + sub);
      for (int i = c0 + lane; i <= c1; i += 32)
        ms = fmaxf(ms, all_ml[(2u * i + (i == c0 ? 1u : 0u)) * p.rows + local].x);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, off));
      const float ref = ms == -INFINITY ? 0.f : ms;
      for (int i = c0 + sub; i <= c1; i += kParts * kSplit) {
        if (i > c0 + sub) fetch(i);
#pragma unroll
        for (int z = 0; z < kParts; ++z) {
          const float w = ml[z].y == 0.f ? 0.f : exp2f(ml[z].x - ref);
          l = fmaf(w, ml[z].y, l);
#pragma unroll
          for (int h = 0; h < kCols; ++h) {
            o[h].x = fmaf(w, y[z][h].x, o[h].x);
            o[h].y = fmaf(w, y[z][h].y, o[h].y);
            o[h].z = fmaf(w, y[z][h].z, o[h].z);
            o[h].w = fmaf(w, y[z][h].w, o[h].w);
          }
        }
      }
    }
    if (kSplit > 1) {
      __syncthreads();
#pragma unroll
      for (int h = 0; h < kCols; ++h) sums[warp][h][lane] = o[h];
      if (lane == 0) sum_l[warp] = l;
      __syncthreads();
      if (sub == 0) {
        for (int z = 1; z < kSplit; ++z) {
          l += sum_l[warp + z];
#pragma unroll
          for (int h = 0; h < kCols; ++h) {
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
      E* dst = static_cast<E*>(a.out) + (q0 + local) * c.d;
#pragma unroll
      for (int h = 0; h < kCols; ++h) {
        const int col = 4 * (lane + 32 * h);
        if (col < c.d) store4(dst + col, make_float4(o[h].x * inv, o[h].y * inv, o[h].z * inv, o[h].w * inv));
      }
      if (lane == 0) a.lse[q0 + local] = l == 0.f ? -INFINITY : (ms + log2f(l)) * kLn2F;
    }
  }
}

// The same for parts of the many-row kernel: a warp takes 32 rows, one to a
// lane, and 4 kQuads columns of them, so that its loads are whole lines.  It
// keeps a running reference as the attention does, so that no pass over the
// parts' maxima comes first.  The row-by-row order took 4.7 us more for 8 units
// of 256 rows over 64 CTAs (28.8 -> 22.7 us, most of it in the writes: a store
// of 32 rows meets 32 lines), and 6 of 98 for 8 trees of 32 drafts.
template <int kSplit, int kQuads, int kParts>
__global__ void __launch_bounds__(kJoinWarps * 32)
    cache_tree_join_kernel(const __grid_constant__ CacheAttnArgs a,
                           const __grid_constant__ AttnPlan p, bool by_unit) {
  __shared__ DivisionShared sh;
  __shared__ float4 sums[kSplit > 1 ? kJoinWarps : 1][kQuads][32];
  __shared__ float2 sum_ml[kSplit > 1 ? kJoinWarps : 1][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = warp % kSplit;
  Shared j;
  if (!shared_unit(a, p, by_unit, sh, j)) return wait_for_parts();
  const int item = blockIdx.x * (kJoinWarps / kSplit) + warp / kSplit;
  const int quads = a.c.d / 4, quad = item % (quads / kQuads) * kQuads;
  const int local = item / (quads / kQuads) * 32 + lane;
  const bool here = local < j.some;
  // rows of all slots: fewer than 2^17, of d floats each
  const float2* all_ml = reinterpret_cast<const float2*>(slot_ml(a, p, 0)) + local;
  const float4* all_o = reinterpret_cast<const float4*>(slot_o(a, p, 0)) + quad * p.rows + local;
  const uint32_t rows = p.rows;
  wait_for_parts();
  float m = -INFINITY, l = 0.f;
  float4 o[kQuads];
#pragma unroll
  for (int h = 0; h < kQuads; ++h) o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
  // o += w y, l += w x, in a state that holds the reference m
  auto add = [&](float w, float x, const float4 (&y)[kQuads]) {
    l = fmaf(w, x, l);
#pragma unroll
    for (int h = 0; h < kQuads; ++h) {
      o[h].x = fmaf(w, y[h].x, o[h].x);
      o[h].y = fmaf(w, y[h].y, o[h].y);
      o[h].z = fmaf(w, y[h].z, o[h].z);
      o[h].w = fmaf(w, y[h].w, o[h].w);
    }
  };
  auto scale = [&](float w) {
    l *= w;
#pragma unroll
    for (int h = 0; h < kQuads; ++h)
      o[h] = make_float4(o[h].x * w, o[h].y * w, o[h].z * w, o[h].w * w);
  };
  if (here) {
    for (int i = j.c0 + sub; i <= j.c1; i += kParts * kSplit) {
      float2 ml[kParts];
      float4 y[kParts][kQuads];
#pragma unroll
      for (int z = 0; z < kParts; ++z) {
        const int part = i + z * kSplit;
        const bool real = part <= j.c1;
        const uint32_t at = real ? (2u * part + (part == j.c0 ? 1u : 0u)) * rows : 0u;
        ml[z] = real ? all_ml[at] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int h = 0; h < kQuads; ++h)
          y[z][h] = real ? all_o[at * quads + h * rows] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float top = m;
#pragma unroll
      for (int z = 0; z < kParts; ++z) top = fmaxf(top, ml[z].x);
      if (i > j.c0 + sub && top > m) scale(exp2f(m - top));
      m = top;
#pragma unroll
      for (int z = 0; z < kParts; ++z) add(ml[z].y == 0.f ? 0.f : exp2f(ml[z].x - m), ml[z].y, y[z]);
    }
  }
  if (kSplit > 1) {
#pragma unroll
    for (int h = 0; h < kQuads; ++h) sums[warp][h][lane] = o[h];
    sum_ml[warp][lane] = make_float2(m, l);
    __syncthreads();
    if (sub != 0) return;
    float top = m;
    for (int z = 1; z < kSplit; ++z) top = fmaxf(top, sum_ml[warp + z][lane].x);
    if (top > m) scale(exp2f(m - top));
    m = top;
    for (int z = 1; z < kSplit; ++z) {
      const float2 ml = sum_ml[warp + z][lane];
      float4 y[kQuads];
#pragma unroll
      for (int h = 0; h < kQuads; ++h) y[h] = sums[warp + z][h][lane];
      add(ml.y == 0.f ? 0.f : exp2f(ml.x - m), ml.y, y);
    }
  }
  if (!here) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (j.q0 + local) * a.c.d + 4 * quad;
#pragma unroll
  for (int h = 0; h < kQuads; ++h)
    store4(dst + 4 * h, make_float4(o[h].x * inv, o[h].y * inv, o[h].z * inv, o[h].w * inv));
  if (quad == 0) a.lse[j.q0 + local] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2F;
}

template <int kSplit, int kQuads, int kParts>
cudaError_t tree_join_t(const CacheAttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  const int64_t rows = head_rows(a) < p.rows ? head_rows(a) : p.rows;
  const int64_t units = static_cast<int64_t>(a.c.B) * p.div.units, borders = p.div.ctas - 1;
  const bool by_unit = units <= borders;
  const int64_t items = (rows + 31) / 32 * (a.c.d / (4 * kQuads));
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((items * kSplit + kJoinWarps - 1) / kJoinWarps),
                     static_cast<unsigned>(by_unit ? units : borders));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_tree_join_kernel<kSplit, kQuads, kParts>, a, p, by_unit);
}

template <typename E, int kSplit, int kCols>
cudaError_t join_t(const CacheAttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  constexpr int kStep = kJoinWarps / kSplit;
  const int64_t rows = head_rows(a) < p.rows ? head_rows(a) : p.rows;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // A block waits for its parts, so it takes rows one after another only where
  // there would be more blocks than the SMs hold at once.
  const int64_t steps = (rows + kStep - 1) / kStep;
  const int64_t units = static_cast<int64_t>(a.c.B) * p.div.units, borders = p.div.ctas - 1;
  const bool by_unit = units <= borders;
  const int64_t held = static_cast<int64_t>(device_sm_count()) * 8;
  const int64_t passes = (steps * (by_unit ? units : borders) + held - 1) / held;
  const int block_rows = static_cast<int>(passes) * kStep;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + block_rows - 1) / block_rows),
                     static_cast<unsigned>(by_unit ? units : borders));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<E, kSplit, kCols>, a, p, block_rows, by_unit);
}

template <int kSplit>
cudaError_t join_s(const CacheAttnArgs& a, const AttnPlan& p, bool bf16, cudaStream_t s) {
  if (a.c.d <= 128)
    return bf16 ? join_t<__nv_bfloat16, kSplit, 1>(a, p, s) : join_t<float, kSplit, 1>(a, p, s);
  return bf16 ? join_t<__nv_bfloat16, kSplit, 2>(a, p, s) : join_t<float, kSplit, 2>(a, p, s);
}

template <typename H, typename F>
cudaError_t launch_ffma_t(const CacheAttnArgs& a, int ctas, cudaStream_t s) {
  AttnPlan p;
  p.rows = F::kRows;
  p.row_tiles = static_cast<int>((head_rows(a) + F::kRows - 1) / F::kRows);
  p.div.units = a.c.heads * p.row_tiles;
  p.div.tile = F::kTile;
  p.div.ctas = ctas;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    const int most = F::smem(RA_MAX_HEAD_DIM);
    e = cudaFuncSetAttribute(cache_attn_ffma_kernel<H, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             most < kFfmaSmem ? most : kFfmaSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cache_attn_ffma_kernel<H, F><<<p.div.ctas, F::kThreads, F::smem(a.c.d), s>>>(a, p);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_cache_attn_join(a, p, false, s) : e;
}

template <typename H, int NC>
cudaError_t launch_ffma(const CacheAttnArgs& a, cudaStream_t s) {
  const int64_t rows = head_rows(a);
  // The smallest group of rows that holds a head's, with as many warps on the
  // keys as leave room for three CTAs on an SM.  Groups of 64 rows feed more
  // products from a read, but groups of 16 keep four CTAs on an SM and none of
  // their rows idle: the latter are ahead until a head has `few` rows (2 heads, 4
  // or 32 sequences of 4000, us with groups of 16 and of 64: d = 64, 40 rows 37
  // 43 / 135 124, 64 rows 41 48 / 181 143; d = 128, 64 rows 58 84 / 279 285, 96
  // rows 76 107 / 408 502, 128 rows 92 119 / 548 530; d = 176, 40 rows 93 96 / 456
  // 322; one tile of d = 240, 18 rows 22 49).
  const int few = a.c.d > 128 ? 32 : a.c.d > 64 ? 96 : 48;
  using F4 = Ffma<4, 1, 1, 4, NC>;
  using F8 = Ffma<4, 1, 2, 2, NC>;
  using F16 = Ffma<4, 1, 4, 1, NC>;
  using F64 = Ffma<8, 2, 8, 1, NC>;
  constexpr int third = kFfmaSmem / 3;
  if (rows <= 4 && F4::smem(a.c.d) <= third) return launch_ffma_t<H, F4>(a, kFfmaCtas, s);
  if (rows <= 8 && F8::smem(a.c.d) <= third) return launch_ffma_t<H, F8>(a, kFfmaCtas, s);
  if (rows <= few || F64::smem(a.c.d) > kFfmaSmem) return launch_ffma_t<H, F16>(a, kFfmaCtas, s);
  return launch_ffma_t<H, F64>(a, kFfmaCtas / 2, s);
}

}  // namespace

cudaError_t launch_cache_attn_join(const CacheAttnArgs& a, const AttnPlan& p, bool bf16,
                                   cudaStream_t s) {
  // A unit is shared by about ctas / units CTAs, and a row's parts are taken
  // four at a time.  Several warps for a row shorten that chain, but then there
  // are more blocks, and a block's own start costs as much as a round or two
  // (8 units of 128 rows over 152 CTAs, the whole call: 1, 2, 4, 8 warps 77.8,
  // 78.6, 81.9, 82.7 us; 1 unit over 304 CTAs, 1 row: 2 or 8 warps 27.6, 20.2 us).
  const int64_t units = static_cast<int64_t>(a.c.B) * p.div.units;
  if (p.div.ctas > 48 * units) return join_s<8>(a, p, bf16, s);
  if (p.div.ctas > 16 * units) return join_s<2>(a, p, bf16, s);
  return join_s<1>(a, p, bf16, s);
}

cudaError_t launch_cache_tree_join(const CacheAttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  // Many parts: warps share them.  Few: many units or borders, so fewer and
  // larger blocks (12 sequences of 552 rows, 9 heads: 4 column quads a warp 78
  // us, 1 quad 90; one unit of 120 rows over 152 CTAs: 8 warps a row 29 us).
  const int64_t units = static_cast<int64_t>(a.c.B) * p.div.units;
  if (p.div.ctas > 32 * units) return tree_join_t<8, 1, 4>(a, p, s);
  if (p.div.ctas > 8 * units) return tree_join_t<2, 2, 4>(a, p, s);
  return tree_join_t<1, 4, 2>(a, p, s);
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a, ra_dtype dense, ra_dtype held,
                                   cudaStream_t s) {
  if (dense == RA_F32)
    return a.c.d <= 128 ? (held == RA_E4M3 ? launch_ffma<__nv_fp8_e4m3, 2>(a, s) : launch_ffma<float, 2>(a, s))
                        : (held == RA_E4M3 ? launch_ffma<__nv_fp8_e4m3, 4>(a, s) : launch_ffma<float, 4>(a, s));
  // The decode kernel reads a key head once per 16 query rows, the tree kernel
  // once per 256.  Up to 16 rows the former is ahead throughout.  With 17 to 32
  // rows it still is over 8-bit caches at d = 128, which the tree kernel has to
  // widen (8 heads, 32 rows, 16 sequences of 16384: 192 against 227 us, 2 of
  // 60000: 102 against 115; bf16: 331 against 183 for the former), and even at d =
  // 64 (141 against 133, 72 against 73).
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
  int64_t most = kFfmaCtas * 16;
  if (rows > 16) most = kTreeCtas * (rows > 128 ? 256 : 128);
  return 2 * most * (d + 2) * 4;
}

}  // namespace ra
