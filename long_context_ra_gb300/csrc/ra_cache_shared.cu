// Attention of new tokens over a paged cache, of sequences that share prefixes
// (samples or beams of one context, one instruction before many requests): a
// prefix is brought in once for all of a group's queries.
//
// With (m, l, o) the online-softmax state of a row over a set of keys, the
// state over all keys is the join of that over the prefix and that over the
// rest, so the two can be worked on by launches of unlike shape: the prefix by
// the rows of up to tile x members sequences at once, which puts a decode step
// on the tensor cores; a sequence's own part as before.  Both run the kernels
// of ra_cache_attention over a list of stretches (ra_paged.cuh), so that
// pages, types, masks, the division of ragged work and the parts of shared
// units are theirs.  Four launches, each behind the one before:
//   plan     one block: groups, their common tokens, the two lists
//   prefix   one stretch per group and lot of members
//   own      one stretch per sequence
//   join     every query row from its states, in order
// A group's common part is cut to whole key tiles and pages, so no tile of it
// holds a draft or an end, and a sequence's own part begins at a page.

#include "ra_cache_attn.cuh"

namespace ra {
namespace {

constexpr int kPlanThreads = 1024;    // at most
constexpr int kPlanSequences = 2048;  // 20 bytes of shared memory each
constexpr int kTile = 128;            // a multiple of every kernel's key tile
constexpr int kLeadKeys = 512;        // keys that take a CTA as long as a unit's start and end

// The plan in the workspace.
struct Plan {
  Stretch* list[2];   // [B] prefixes; [B] own parts, one per sequence
  int64_t* at[2];     // lengths before each
  int64_t* totals;    // [2][2] length of all; stretches
  int32_t* lot;       // [B] the prefix stretch that a sequence is a member of, or -1
};

struct PlanArgs {
  PagedArgs c;
  const int32_t* shared;
  Plan plan;
  int tile[2];      // keys per tile of the two launches
  int lead[2];
  int granule;      // a common part is a multiple of it
  int members;      // sequences of a lot
};

// Inclusive scan of two values per thread over the block; `all`: the sums.
__device__ __forceinline__ longlong2 scan_two(longlong2 x, longlong2* warps, longlong2& all) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  auto scan = [&](longlong2 v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, v.x, o), b = __shfl_up_sync(0xffffffffu, v.y, o);
      if (lane >= o) v.x += a, v.y += b;
    }
    return v;
  };
  x = scan(x);
  __syncthreads();
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  const longlong2 w = scan(lane * 32 < static_cast<int>(blockDim.x) ? warps[lane] : longlong2{0, 0});
  all.x = __shfl_sync(0xffffffffu, w.x, 31);
  all.y = __shfl_sync(0xffffffffu, w.y, 31);
  const int64_t bx = __shfl_sync(0xffffffffu, w.x, max(warp - 1, 0)), by = __shfl_sync(0xffffffffu, w.y, max(warp - 1, 0));
  if (warp > 0) x.x += bx, x.y += by;
  return x;
}

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int32_t smem[];
  __shared__ longlong2 warps[32];
  const PagedArgs& c = a.c;
  const int B = c.B, tid = threadIdx.x;
  const int G = B + 1;           // groups: 0 for live sequences ahead of the first that shares nothing
  int32_t* group = smem;         // [B] group of each sequence
  int32_t* common = group + B;   // [G] tokens in common, then the shared part
  int32_t* first = common + G;   // [G] its first and last live sequence
  int32_t* last = first + G;
  int32_t* lots = last + G;      // [G] live sequences, then the first lot
  allow_join();
  for (int i = tid; i < G; i += blockDim.x) {
    common[i] = INT32_MAX;
    first[i] = B;
    last[i] = -1;
    lots[i] = 0;
  }
  const int each = (B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(B, tid * each), b1 = min(B, b0 + each);
  // ---- groups: one begins where a live sequence shares nothing
  longlong2 sum{0, 0}, all;
  for (int b = b0; b < b1; ++b) sum.x += c.lens[b] >= 0 && a.shared[b] <= 0;
  int64_t at = scan_two(sum, warps, all).x - sum.x;
  for (int b = b0; b < b1; ++b) {
    const bool live = c.lens[b] >= 0;
    at += live && a.shared[b] <= 0;
    const int g = static_cast<int>(at);
    group[b] = g;
    if (live) {
      atomicMin(first + g, b);
      atomicMax(last + g, b);
      atomicAdd(lots + g, 1);
      if (c.count && c.count[b] > c.T) flag_page(c.status);
    }
  }
  __syncthreads();
  for (int b = b0; b < b1; ++b)
    if (c.lens[b] >= 0) atomicMin(common + group[b], b == first[group[b]] ? c.lens[b] : min(c.lens[b], a.shared[b]));
  __syncthreads();
  // ---- their shared parts and lots of members
  const int g1 = b0 < B && b1 == B ? G : b1;
  sum = longlong2{0, 0};
  for (int g = b0; g < g1; ++g) {
    const int part = lots[g] > 1 ? max(common[g], 0) / a.granule * a.granule : 0;
    const int n = part > 0 ? (last[g] - first[g] + a.members) / a.members : 0;
    common[g] = part;
    lots[g] = n;
    sum.x += n;
    sum.y += n * stretch_length(part / a.tile[0], a.lead[0]);
  }
  longlong2 before = scan_two(sum, warps, all);
  before.x -= sum.x;
  before.y -= sum.y;
  for (int g = b0; g < g1; ++g) {
    const int n = lots[g];
    lots[g] = static_cast<int>(before.x);
    for (int i = 0; i < n; ++i) {
      const int b = first[g] + i * a.members;
      a.plan.list[0][before.x] = Stretch{common[g], 0, first[g], 0, b, min(a.members, last[g] + 1 - b)};
      a.plan.at[0][before.x] = before.y;
      before.x += 1;
      before.y += stretch_length(common[g] / a.tile[0], a.lead[0]);
    }
  }
  if (tid == 0) {
    a.plan.totals[0] = all.y;
    a.plan.totals[1] = all.x;
  }
  __syncthreads();
  // ---- own parts
  sum = longlong2{0, 0};
  auto own = [&](int b) {
    const SeqInfo s = sequence(c, b);
    const int part = c.lens[b] >= 0 ? common[group[b]] : 0;
    return Stretch{static_cast<int32_t>(s.len) - part, s.cnt, b, part >> c.page_shift, b, 1};
  };
  auto length = [&](const Stretch& s) {
    return stretch_length(stretch_tiles(SeqInfo{s.len, s.cnt}, a.tile[1]), a.lead[1]);
  };
  for (int b = b0; b < b1; ++b) sum.x += length(own(b));
  int64_t own_at = scan_two(sum, warps, all).x - sum.x;
  for (int b = b0; b < b1; ++b) {
    const Stretch s = own(b);
    a.plan.list[1][b] = s;
    a.plan.at[1][b] = own_at;
    own_at += length(s);
    const int g = group[b];
    a.plan.lot[b] = c.lens[b] >= 0 && common[g] > 0 ? lots[g] + (b - first[g]) / a.members : -1;
  }
  if (tid == 0) {
    a.plan.totals[2] = all.x;
    a.plan.totals[3] = B;
  }
}

// ------------------------------------------------------------------- join
// A lane has a row and 4 kQuads columns of it: a warp's 32 rows make whole lines
// of states laid out a column quad of all rows at a time.
struct Side {
  const Stretch* list;
  const int64_t* at;
  const int64_t* totals;
  const float2* part_ml;   // [slots][rows]
  const float4* part_o;    // a slot's rows x d / 4 quads
  const float2* whole_ml;
  const float4* whole_o;
  int rows, ctas, tile, lead, tile_members, tile_rows;
  int row_step, quad_step;  // of a slot's quads
};

struct JoinArgs {
  CacheAttnArgs a;
  Side side[2];
  const int32_t* lot;
  int64_t all_rows;
  int32_t rows1;
};

constexpr int kJoinThreads = 128;
constexpr int kQuads = 2;
constexpr int kParts = 4;

template <typename E, int kSplit>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const __grid_constant__ JoinArgs j) {
  constexpr int kItems = kJoinThreads / 32 / kSplit;  // of a block
  __shared__ float4 sums[kSplit > 1 ? kJoinThreads / 32 : 1][kQuads][32];
  __shared__ float2 sum_ml[kSplit > 1 ? kJoinThreads / 32 : 1][32];
  const CacheAttnArgs& a = j.a;
  const PagedArgs& c = a.c;
  const int quads = c.d / 4, slices = quads / kQuads;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = warp % kSplit;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kItems + warp / kSplit;
  const int quad = static_cast<int>(item % slices) * kQuads;
  const int64_t row = item / slices * 32 + lane;
  const bool here = row < j.all_rows;
  wait_for_parts();
  const int w = static_cast<int>(row % j.rows1);  // within its sequence and key head
  const int head = static_cast<int>(row / j.rows1 % c.heads);
  const int b = static_cast<int>(row / j.rows1 / c.heads);
  float m = -INFINITY, l = 0.f;
  float4 o[kQuads];
#pragma unroll
  for (int h = 0; h < kQuads; ++h) o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto scale = [&](float f) {
    l *= f;
#pragma unroll
    for (int h = 0; h < kQuads; ++h) o[h] = make_float4(o[h].x * f, o[h].y * f, o[h].z * f, o[h].w * f);
  };
  if (here && w % c.T < sequence(c, b).cnt) {
#pragma unroll 1
    for (int z = 0; z < 2; ++z) {
      const Side& s = j.side[z];
      const int v = z == 0 ? j.lot[b] : b;
      if (v < 0) continue;
      const Stretch st = s.list[v];
      const int64_t tiles = stretch_tiles(SeqInfo{st.len, st.cnt}, s.tile);
      const int64_t run = (s.totals[0] * c.heads + s.ctas - 1) / s.ctas;
      const int64_t u0 = s.at[v] * c.heads + head * stretch_length(tiles, s.lead);
      const int c0 = static_cast<int>(u0 / run), c1 = static_cast<int>((u0 + tiles - 1) / run);
      const int member = b - st.b0;
      const int local = member / s.tile_members * s.tile_rows + member % s.tile_members * j.rows1 + w;
      const bool whole = c0 == c1;
      const float2* ml_at = whole ? s.whole_ml + row : s.part_ml + local;
      const float4* o_at = whole ? s.whole_o + quad * j.all_rows + row : s.part_o + quad * s.quad_step + local * s.row_step;
      const int64_t quad_step = whole ? j.all_rows : s.quad_step;
      // the own part's few by the last warp, the prefix's from the first on
      for (int i = c0 + (z == 0 ? sub : kSplit - 1 - sub) * kParts; i <= c1; i += kParts * kSplit) {
        float2 ml[kParts];
        float4 y[kParts][kQuads];
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
          const bool real = i + x <= c1;
          const int64_t slot = whole ? 0 : (2 * (i + x) + (i + x == c0 ? 1 : 0));
          ml[x] = real ? ml_at[slot * s.rows] : make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int h = 0; h < kQuads; ++h)
            y[x][h] = real ? o_at[slot * s.rows * quads + h * quad_step] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float top = m;
#pragma unroll
        for (int x = 0; x < kParts; ++x) top = fmaxf(top, ml[x].x);
        if (top > m && m > -INFINITY) scale(exp2f(m - top));
        m = top;
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
          // a weight of 0 multiplies too: o may be NaN, and is 0 without a seen key
          const float f = ml[x].y == 0.f ? 0.f : exp2f(ml[x].x - m);
          l = fmaf(f, ml[x].y, l);
#pragma unroll
          for (int h = 0; h < kQuads; ++h) {
            o[h].x = fmaf(f, y[x][h].x, o[h].x);
            o[h].y = fmaf(f, y[x][h].y, o[h].y);
            o[h].z = fmaf(f, y[x][h].z, o[h].z);
            o[h].w = fmaf(f, y[x][h].w, o[h].w);
          }
        }
      }
    }
  }
  if (kSplit > 1) {
#pragma unroll
    for (int h = 0; h < kQuads; ++h) sums[warp][h][lane] = o[h];
    sum_ml[warp][lane] = make_float2(m, l);
    __syncthreads();
    if (sub != 0) return;
    float top = m;
#pragma unroll
    for (int z = 1; z < kSplit; ++z) top = fmaxf(top, sum_ml[warp + z][lane].x);
    if (top > m && m > -INFINITY) scale(exp2f(m - top));
    m = top;
#pragma unroll
    for (int z = 1; z < kSplit; ++z) {
      const float2 ml = sum_ml[warp + z][lane];
      const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - m);
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int h = 0; h < kQuads; ++h) {
        const float4 y = sums[warp + z][h][lane];
        o[h].x = fmaf(f, y.x, o[h].x);
        o[h].y = fmaf(f, y.y, o[h].y);
        o[h].z = fmaf(f, y.z, o[h].z);
        o[h].w = fmaf(f, y.w, o[h].w);
      }
    }
  }
  if (!here) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  E* dst = static_cast<E*>(a.out) + row * c.d + 4 * quad;
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int h = 0; h < kQuads; ++h)
      reinterpret_cast<float4*>(dst)[h] = make_float4(o[h].x * inv, o[h].y * inv, o[h].z * inv, o[h].w * inv);
  } else {
    uint32_t x[2 * kQuads];
#pragma unroll
    for (int h = 0; h < kQuads; ++h) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(o[h].x * inv, o[h].y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(o[h].z * inv, o[h].w * inv);
      x[2 * h] = *reinterpret_cast<const uint32_t*>(&lo);
      x[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&hi);
    }
    static_assert(kQuads == 2, "16 bytes of bf16");
    *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
  }
  if (quad == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2F;
}

template <typename E, int kSplit>
cudaError_t join(const JoinArgs& j, int64_t items, cudaStream_t s) {
  constexpr int kItems = kJoinThreads / 32 / kSplit;
  const dim3 grid(static_cast<unsigned>((items + kItems - 1) / kItems));
  return launch_behind(shared_join_kernel<E, kSplit>, grid, kJoinThreads, 0, s, j);
}

// ------------------------------------------------------------ the workspace
constexpr int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

struct Room {
  int64_t plan, parts[2], whole[2], end;
};

// Slot rows of the two launches, for the largest kernel that may take them.
Room room(int32_t B, int64_t rows1, int32_t heads, int32_t d) {
  const int64_t all = B * rows1 * heads;
  const int64_t slots = 2ll * (B * rows1 > 16 ? kTreeCtas * 256 : kFfmaCtas * 16);
  const int64_t own = 2ll * (rows1 > 16 ? kTreeCtas * 128 : kFfmaCtas * 16);
  Room r;
  r.plan = 0;
  r.parts[0] = round256(static_cast<int64_t>(B) * (2 * sizeof(Stretch) + 2 * 8 + 4) + 4 * 8 + 5 * 256);
  r.parts[1] = r.parts[0] + round256(slots * (d + 2) * 4);
  r.whole[0] = r.parts[1] + round256(own * (d + 2) * 4);
  r.whole[1] = r.whole[0] + round256(all * (d + 2) * 4 + 256);
  r.end = r.whole[1] + round256(all * (d + 2) * 4 + 256);
  return r;
}

}  // namespace

int64_t cache_attention_shared_workspace_bytes(int32_t B, int32_t Hq, int32_t heads, int32_t T, int32_t d) {
  const int64_t plain = cache_attention_workspace_bytes(B, Hq, heads, T, d);
  const int64_t shared = room(B, static_cast<int64_t>(Hq / heads) * T, heads, d).end;
  return plain > shared ? plain : shared;
}

cudaError_t launch_cache_attention_shared(const CacheAttnArgs& a, const int32_t* shared, ra_dtype dense,
                                          ra_dtype held, cudaStream_t s) {
  const int64_t rows1 = head_rows(a), stacked = a.c.B * rows1;
  const bool k8 = held == RA_E4M3;
  // The kernel for a lot's rows, by all rows that there may be, and the one for
  // a sequence's own.
  SharedKernel kernel[2];
  SharedShape shape[2];
  if (dense == RA_F32) {
    for (int z = 0; z < 2; ++z) {
      kernel[z] = ffma_kernel(z == 0 ? stacked : rows1, a.c.d);
      shape[z] = ffma_shape(kernel[z]);
    }
  } else {
    kernel[0] = stacked > 128 ? SharedKernel::kTreeTwo : stacked > kDecodeRows ? SharedKernel::kTreeOne
                                                                              : SharedKernel::kDecode;
    kernel[1] = rows1 > kDecodeRows ? SharedKernel::kTreeOne : SharedKernel::kDecode;
    for (int z = 0; z < 2; ++z)
      shape[z] = kernel[z] == SharedKernel::kDecode ? decode_shape()
                                                    : tree_shape(a.c.d, kernel[z] == SharedKernel::kTreeTwo);
  }
  const int64_t tile_members = rows1 > 0 ? shape[0].tile_rows / rows1 : 0;
  const int64_t members = tile_members * (shape[0].rows / shape[0].tile_rows);
  // Nothing to gain where a unit has no room for a second sequence's rows.
  if (a.c.B < 2 || a.c.B > kPlanSequences || members < 2 || rows1 > shape[1].rows)
    return launch_cache_attention(a, dense, held, s);

  const int B = a.c.B;
  const Room r = room(B, rows1, a.c.heads, a.c.d);
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.ws);
  PlanArgs pl;
  pl.c = a.c;
  pl.shared = shared;
  uint8_t* at = ws + r.plan;
  auto take = [&](int64_t bytes) {
    uint8_t* x = at;
    at += round256(bytes);
    return x;
  };
  pl.plan.totals = reinterpret_cast<int64_t*>(take(4 * 8));
  for (int z = 0; z < 2; ++z) {
    pl.plan.list[z] = reinterpret_cast<Stretch*>(take(B * sizeof(Stretch)));
    pl.plan.at[z] = reinterpret_cast<int64_t*>(take(B * 8));
    pl.tile[z] = shape[z].tile;
    pl.lead[z] = kLeadKeys / shape[z].tile;
  }
  pl.plan.lot = reinterpret_cast<int32_t*>(take(B * 4));
  const int page = 1 << a.c.page_shift;
  pl.granule = page > kTile ? page : kTile;
  pl.members = static_cast<int>(members);
  const int threads = B < kPlanThreads ? (B + 31) / 32 * 32 : kPlanThreads;  // fewer warps are quicker
  shared_plan_kernel<<<1, threads, B * 20 + 16, s>>>(pl);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  JoinArgs j;
  j.a = a;
  j.lot = pl.plan.lot;
  j.all_rows = static_cast<int64_t>(B) * a.c.heads * rows1;
  j.rows1 = static_cast<int32_t>(rows1);
  for (int z = 0; z < 2; ++z) {
    SharedAttnArgs g;
    static_cast<CacheAttnArgs&>(g) = a;
    g.ws = reinterpret_cast<float*>(ws + r.parts[z]);
    static_cast<PagedArgs&>(g.stretches) = a.c;
    g.stretches.list = pl.plan.list[z];
    g.stretches.at = pl.plan.at[z];
    g.stretches.totals = pl.plan.totals + 2 * z;
    g.stretches.lead = pl.lead[z];
    g.whole_o = reinterpret_cast<float*>(ws + r.whole[z]);
    g.whole_ml = g.whole_o + round256(j.all_rows * a.c.d * 4) / 4;
    g.all_rows = j.all_rows;
    g.rows1 = j.rows1;
    g.tile_members = static_cast<int32_t>(z == 0 ? tile_members : 1);
    AttnPlan p;
    p.div = Division{a.c.heads, shape[z].tile, shape[z].ctas};
    p.rows = shape[z].rows;
    p.row_tiles = 1;
    if (kernel[z] == SharedKernel::kDecode)
      e = launch_shared_decode(g, p, k8, s);
    else if (kernel[z] == SharedKernel::kTreeOne || kernel[z] == SharedKernel::kTreeTwo)
      e = launch_shared_tree(g, p, k8, s);
    else
      e = launch_shared_ffma(g, p, kernel[z], k8, s);
    if (e != cudaSuccess) return e;
    const float* parts = g.ws;
    const int64_t slots = 2ll * p.div.ctas;
    j.side[z] = Side{g.stretches.list,
                     g.stretches.at,
                     g.stretches.totals,
                     reinterpret_cast<const float2*>(parts),
                     reinterpret_cast<const float4*>(parts + slots * p.rows * 2),
                     reinterpret_cast<const float2*>(g.whole_ml),
                     reinterpret_cast<const float4*>(g.whole_o),
                     p.rows,
                     p.div.ctas,
                     p.div.tile,
                     pl.lead[z],
                     g.tile_members,
                     shape[z].tile_rows,
                     shape[z].quads ? 1 : a.c.d / 4,
                     shape[z].quads ? p.rows : 1};
  }
  // Four warps to a row's parts where those of a single group may be many.
  const int64_t items = (j.all_rows + 31) / 32 * (a.c.d / 4 / kQuads);
  const int64_t units = a.c.heads * ((B + members - 1) / members);
  const bool many = shape[0].ctas > 8 * units;
  if (dense == RA_BF16) return many ? join<__nv_bfloat16, 4>(j, items, s) : join<__nv_bfloat16, 1>(j, items, s);
  return many ? join<float, 4>(j, items, s) : join<float, 1>(j, items, s);
}

}  // namespace ra
