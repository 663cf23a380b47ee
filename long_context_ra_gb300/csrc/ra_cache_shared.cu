// Attention of new tokens over a paged cache, of sequences that share prefixes
// (samples or beams of one context, one instruction before many requests): a
// prefix is brought in once for all of a group's queries.
//
// With (m, l, o) the online-softmax state of a row over a set of keys, the
// state over all keys is the join of that over the prefix and that over the
// rest, so the two can be worked on by units of unlike shape: the prefix by the
// new tokens' rows of all of a group's sequences, laid end to end and cut into
// lots, which puts a decode step on the tensor cores; a sequence's own part as
// before.  Both run the kernels of ra_cache_attention over a list of stretches
// (ra_paged.cuh), so that pages, types, masks, the division of ragged work and
// the parts of shared units are theirs.  The launches, one behind the other (one
// that may begin ahead of its turn takes SMs from the one before it: 64 samples of
// 16384 tokens 93 us where all may, 78 where none does):
//   plan      one block: groups, their common tokens, the rows, the stretches
//   prefixes  a stretch per lot of a group
//   own parts a stretch per sequence (in one launch with the prefixes where the
//             same kernel takes both)
//   join      every query row from its states, in order
// A group's common part is cut to whole key tiles and pages, so no tile of it
// holds a draft or an end, and a sequence's own part begins at a page.

#include "ra_cache_attn.cuh"

namespace ra {
namespace {

constexpr int kPlanThreads = 1024;    // at most
constexpr int kPlanSequences = 2048;  // 32 bytes of shared memory each
constexpr int kTile = 128;            // a multiple of every kernel's key tile
constexpr int kMostRows = 256;        // of a lot in any kernel
// Bytes of the table of all sequences but one below which prefixes are read again,
// as plan, second launch and join take some 20 us and short units more.  The host
// sees the table's width alone, so the rule fits tables about as wide as the
// sequences are long (at worst 8 us off below: 4 of 16384 out of 8 bits) and shares
// too much in wider ones.  (us shared, not shared, replayed graphs, tails of 100, 4
// queries a head, f32 2; MB repeated.  bf16, 8 heads of
// 128: 3 sequences of 1024 27 17; 4 of 4096, 50 MB, 27 25; 4 of 8192, 101 MB, 29 29;
// 4 of 16384, 201 MB, 31 41; 16 of 1024, 63 MB, 39 24; 16 of 2048, 126 MB, 39 29; 16
// of 4096, 252 MB, 40 39; 16 of 8192, 503 MB, 43 58; 64 of 1024, 264 MB, 54 51; 64 of
// 2048, 528 MB, 56 70; 64 of 16384, 70 336.  Out of 8 bits: 4 of 8192, 50 MB, 31 31;
// 4 of 16384, 101 MB, 33 41; 16 of 2048, 63 MB, 41 31; 16 of 4096, 126 MB, 42 40; 16 of
// 8192, 252 MB, 46 62; 64 of 1024, 132 MB, 54 53; 64 of 2048, 264 MB, 56 74.  2 heads of
// 64: 64 of 4096, 132 MB, 38 29; 64 of 8192, 264 MB, 39 41.  f32, 4 heads of 80: 4 of
// 8192, 63 MB, 40 41; 4 of 16384, 126 MB, 45 60; 16 of 2048, 79 MB, 46 39; 16 of 4096,
// 157 MB, 56 60.)  Groups are not weighed one by one: in a batch that shares, a pair
// with a tile in common has a lot of its own.
constexpr int64_t kWorthSharing = 160ll << 20;
constexpr int kRuns = 9;              // lengths of a run that are tried

// Where a sequence's rows are among the lots: row r of its live ones is row
// (rel + r) of lot `lot` on (-1: its group has nothing in common).
struct Place {
  int32_t lot, rel;
};

// The plan in the workspace.  List 1 may be the same as list 0, behind it.
struct Plan {
  Stretch* list[2];
  int64_t* totals;   // [2][3] length of all, stretches, run; then the first own stretch in its list
  Place* places;     // [B]
  int32_t* rows_of;  // [B rows1]
};

struct PlanArgs {
  PagedArgs c;
  const int32_t* shared;
  Plan plan;
  int tile_shift[2];  // log2 of the keys per tile of the two kinds of stretches
  int lead[2];
  int ctas[2];
  int granule;   // a common part is a multiple of it
  int lot_rows, lot_shift;  // query rows of a lot, and their log2
  int group;     // query heads of a key head
  bool one_list;
};

// Inclusive scan of two values per thread over the block; `all`: the sums.
__device__ __noinline__ longlong2 scan_two(longlong2 x, longlong2* warps, longlong2& all) {
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

// One block that runs through its code once: bound by the loads of that code as
// much as by the chain of scans, so that loops stay loops and the scan is a
// function (32 samples, the whole call: 78 us with all of it inlined and unrolled,
// 75 without).
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int32_t smem[];
  __shared__ longlong2 warps[32];
  __shared__ int runs[kRuns], again;
  const PagedArgs& c = a.c;
  const int B = c.B, tid = threadIdx.x;
  const int G = B + 1;           // groups: 0 for live sequences ahead of the first that shares nothing
  int32_t* group = smem;         // [B] group of each sequence
  int32_t* row_at = group + B;   // [B] its first live row among those of the lots
  int32_t* len = row_at + B;     // [B] lens
  int32_t* cnt = len + B;        // [B] new tokens
  int32_t* common = cnt + B;     // [G] tokens in common, then the shared part
  int32_t* first = common + G;   // [G] its first live sequence
  int32_t* rows = first + G;     // [G] live rows
  int32_t* lots = rows + G;      // [G] live sequences, then the first lot
  if (tid < kRuns) runs[tid] = 0;
  if (tid == 0) again = 0;
#pragma unroll 1
  for (int i = tid; i < G; i += blockDim.x) {
    common[i] = INT32_MAX;
    first[i] = B;
    rows[i] = 0;
    lots[i] = 0;
  }
  const int each = (B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(B, tid * each), b1 = min(B, b0 + each);
  const int g1 = b0 < B && b1 == B ? G : b1;  // this thread's groups: b0 .. g1 - 1
  // ---- groups: one begins where a live sequence shares nothing
  longlong2 sum{0, 0}, all;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int n = c.lens[b], t = c.count ? c.count[b] : c.T;
    len[b] = n;
    cnt[b] = n < 0 ? 0 : max(0, min(t, c.T));
    if (n >= 0 && t > c.T) flag_page(c.status);
    group[b] = a.shared[b];
    sum.x += n >= 0 && group[b] <= 0;
  }
  int64_t at = scan_two(sum, warps, all).x - sum.x;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    at += len[b] >= 0 && group[b] <= 0;
    if (len[b] >= 0) {
      atomicMin(first + at, b);
      atomicAdd(lots + at, 1);
    }
    row_at[b] = group[b];  // for the moment
    group[b] = static_cast<int>(at);
  }
  __syncthreads();
#pragma unroll 1
  for (int b = b0; b < b1; ++b)
    if (len[b] >= 0) atomicMin(common + group[b], b == first[group[b]] ? len[b] : min(len[b], row_at[b]));
  __syncthreads();
#pragma unroll 1
  for (int g = b0; g < g1; ++g) common[g] = lots[g] > 1 ? max(common[g], 0) / a.granule * a.granule : 0;
  __syncthreads();
  // ---- rows that see a prefix
  sum = longlong2{0, 0};
  auto live_rows = [&](int b) { return common[group[b]] > 0 ? cnt[b] * a.group : 0; };
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int n = live_rows(b);
    sum.x += n;
    if (n > 0) atomicAdd(rows + group[b], n);
  }
  int row = static_cast<int>(scan_two(sum, warps, all).x - sum.x);
  const int rows_all = static_cast<int>(all.x);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    row_at[b] = row;
    row += live_rows(b);
  }
  __syncthreads();
  // ---- lengths: of a lot's units, and of a sequence's own
  auto lots_of = [&](int g) { return common[g] > 0 ? (rows[g] + a.lot_rows - 1) >> a.lot_shift : 0; };
  auto lot_length = [&](int g) {
    return c.heads * stretch_length(common[g] >> a.tile_shift[0], a.lead[0]);
  };
  auto part = [&](int b) { return cnt[b] > 0 ? common[group[b]] : 0; };
  auto own = [&](int b) { return cnt[b] > 0 ? len[b] - part(b) : 0; };  // without new tokens: nothing
  auto length = [&](int b) {
    const int64_t keys = static_cast<int64_t>(own(b)) + cnt[b];
    return c.heads * stretch_length((keys + (1 << a.tile_shift[1]) - 1) >> a.tile_shift[1], a.lead[1]);
  };
  sum = longlong2{0, 0};
#pragma unroll 1
  for (int g = b0; g < g1; ++g) sum.x += lots_of(g) * lot_length(g);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) sum.y += length(b);
  const longlong2 own_before = scan_two(sum, warps, all);
  int64_t own_at = own_before.y - sum.y;
  const int64_t own_all = all.y, total = all.x + (a.one_list ? own_all : 0);
  // ---- the run of a CTA.  Lots of a group read the same keys: where they begin
  // at runs' starts they do so at the same time, out of L2 (10 lots of 65536 keys,
  // 8 heads: 2.5 GB from memory without).  The smallest run, up to an eighth
  // above the even one, with which every lot can take whole runs.
  const int64_t even = (total + a.ctas[0] - 1) / a.ctas[0];
  const uint32_t even32 = static_cast<uint32_t>(even);
  auto candidate = [&](int i) { return even32 + even32 / (8 * (kRuns - 1)) * i; };
  const bool small = total < (int64_t{1} << 31);  // the products below stay in 32 bits
#pragma unroll 1
  for (int g = b0; g < g1; ++g) {
    const int n = lots_of(g);
    if (n > 1) again = 1;
    if (n > 0 && small)
#pragma unroll 1
      for (int i = 0; i < kRuns; ++i)
        atomicAdd(&runs[i], n * static_cast<int>((static_cast<uint32_t>(lot_length(g)) + candidate(i) - 1) / candidate(i)));
  }
  __syncthreads();
  int64_t run = even;
  bool aligned = false;
#pragma unroll 1
  for (int i = 0; i < kRuns && again && small && !aligned; ++i) {
    const uint32_t r = candidate(i);
    aligned = runs[i] + (a.one_list ? (static_cast<uint32_t>(own_all) + r - 1) / r : 0u) <= static_cast<uint32_t>(a.ctas[0]);
    if (aligned) run = r;
  }
  // ---- lots
  auto lot_room = [&](int g) {
    const int64_t n = lot_length(g);
    return aligned ? (static_cast<uint32_t>(n + run - 1) / static_cast<uint32_t>(run)) * run : n;
  };
  sum = longlong2{0, 0};
#pragma unroll 1
  for (int g = b0; g < g1; ++g) {
    const int n = lots_of(g);
    sum.x += n;
    if (n > 0) sum.y += n * lot_room(g);
  }
  longlong2 before = scan_two(sum, warps, all);
  before.x -= sum.x;
  before.y -= sum.y;
#pragma unroll 1
  for (int g = b0; g < g1; ++g) {
    const int n = lots_of(g);
    lots[g] = static_cast<int>(before.x);
    const int64_t room = n > 0 ? lot_room(g) : 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      a.plan.list[0][before.x] = Stretch{common[g], 0, first[g], 0, row_at[first[g]] + i * a.lot_rows,
                                         min(a.lot_rows, rows[g] - i * a.lot_rows), before.y, room};
      before.x += 1;
      before.y += room;
    }
  }
  const longlong2 prefixes = all;
  __syncthreads();
  // ---- own parts
  Stretch* list = a.one_list ? a.plan.list[0] + prefixes.x : a.plan.list[1];
  if (a.one_list) own_at += prefixes.y;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    list[b] = Stretch{own(b), cnt[b], b, part(b) >> c.page_shift, ~b, a.group * c.T, own_at, length(b)};
    own_at += length(b);
    const int g = group[b];
    a.plan.places[b] = part(b) > 0 ? Place{lots[g], row_at[b] - row_at[first[g]]} : Place{-1, 0};
  }
  if (tid == 0) {
    a.plan.totals[0] = prefixes.y + (a.one_list ? own_all : 0);
    a.plan.totals[1] = prefixes.x + (a.one_list ? B : 0);
    a.plan.totals[2] = run;
    a.plan.totals[3] = own_all;
    a.plan.totals[4] = B;
    a.plan.totals[5] = (own_all + a.ctas[1] - 1) / a.ctas[1];
    a.plan.totals[6] = a.one_list ? prefixes.x : 0;
  }
  // ---- the query rows of the lots: heads of a sequence one after another, its new tokens only
  for (int r = tid; r < rows_all; r += blockDim.x) {
    int lo = 0, hi = B - 1;  // the last sequence whose rows begin at or before r
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (row_at[mid] <= r)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int j = r - row_at[lo], n = cnt[lo];
    a.plan.rows_of[r] = lo * a.group * c.T + j / n * c.T + j % n;
  }
}

// ------------------------------------------------------------------- join
// A lane has a row and 4 kQuads columns of it: a warp's 32 rows make whole lines
// of states laid out a column quad of all rows at a time.
struct Side {
  const Stretch* list;
  const int64_t* run;
  const float2* part_ml;   // [slots][rows]
  const float4* part_o;    // a slot's rows x d / 4 quads
  const float2* whole_ml;
  const float4* whole_o;
  int rows, tile, lead;
  int row_step, quad_step;  // of a slot's quads
};

struct JoinArgs {
  CacheAttnArgs a;
  Side side[2];
  const Place* places;
  const int64_t* first_own;  // stretch of sequence 0 in side 1's list
  int64_t all_rows;
  int32_t rows1, lot_rows;
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
  const int cnt = here ? sequence(c, b).cnt : 0;
  if (w % c.T < cnt) {
    const Place place = j.places[b];
#pragma unroll 1
    for (int z = 0; z < 2; ++z) {
      const Side& s = j.side[z];
      if (z == 0 && place.lot < 0) continue;
      const int rel = place.rel + w / c.T * cnt + w % c.T;
      const int v = z == 0 ? place.lot + rel / j.lot_rows : b + static_cast<int>(*j.first_own);
      const int local = z == 0 ? rel % j.lot_rows : w;
      const Stretch st = s.list[v];
      const int64_t tiles = stretch_tiles(SeqInfo{st.len, st.cnt}, s.tile);
      const int64_t run = *s.run;
      const int64_t u0 = st.at + head * stretch_length(tiles, s.lead);
      const int c0 = static_cast<int>(u0 / run), c1 = static_cast<int>((u0 + tiles - 1) / run);
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
  shared_join_kernel<E, kSplit><<<grid, kJoinThreads, 0, s>>>(j);
  return cudaGetLastError();
}

// ------------------------------------------------------------ the workspace
constexpr int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

// A group has two sequences at least, and all its lots but one are full; the
// smallest lots have 4 rows.
int64_t lots_at_most(int64_t B, int64_t rows1) { return B / 2 + (B * rows1 + 3) / 4; }

struct Room {
  int64_t plan, parts[2], whole[2], end;
};

// Slot rows of the two launches, for the largest kernel that may take them.
Room room(int32_t B, int64_t rows1, int32_t heads, int32_t d) {
  const int64_t all = B * rows1 * heads;
  const int64_t slots = 2ll * (B * rows1 > 16 ? kTreeCtas * 256 : kFfmaCtas * 16);
  const int64_t own = 2ll * kFfmaCtas * 16;  // one launch takes both above 16 rows of a sequence
  Room r;
  r.plan = 0;
  r.parts[0] = round256(static_cast<int64_t>(B) * (2 * sizeof(Stretch) + sizeof(Place)) + all / heads * 4 +
                        lots_at_most(B, rows1) * sizeof(Stretch) + 7 * 8 + 5 * 256);
  r.parts[1] = r.parts[0] + round256(slots * (d + 2) * 4);
  r.whole[0] = r.parts[1] + round256(own * (d + 2) * 4);
  r.whole[1] = r.whole[0] + round256(all * (d + 2) * 4 + 256);
  r.end = r.whole[1] + round256(all * (d + 2) * 4 + 256);
  return r;
}

// Whether any type's units and the plan have room for sequences of such a batch:
// the plain call's workspace serves for the others.
bool may_share(int32_t B, int64_t rows1) { return B >= 2 && B <= kPlanSequences && 2 * rows1 <= kMostRows; }

}  // namespace

int64_t cache_attention_shared_workspace_bytes(int32_t B, int32_t Hq, int32_t heads, int32_t T, int32_t d) {
  const int64_t plain = cache_attention_workspace_bytes(B, Hq, heads, T, d);
  const int64_t rows1 = static_cast<int64_t>(Hq / heads) * T;
  if (!may_share(B, rows1)) return plain;
  const int64_t shared = room(B, rows1, heads, d).end;
  return plain > shared ? plain : shared;
}

cudaError_t launch_cache_attention_shared(const CacheAttnArgs& a, const int32_t* shared, ra_dtype dense,
                                          ra_dtype held, cudaStream_t s) {
  const int B = a.c.B;
  const int64_t rows1 = head_rows(a), stacked = B * rows1;
  const bool k8 = held == RA_E4M3;
  // The kernel for lots, by all rows that there may be, and the one for a
  // sequence's own.  (Out of 8 bits the former rounds probabilities to bf16, 8
  // bits, as its operands are; the decode kernel, with f16's 11, has units of 16
  // rows and would read a prefix again for every 16 of a group's.)
  SharedKernel kernel[2];
  SharedShape shape[2];
  if (dense == RA_F32) {
    for (int z = 0; z < 2; ++z) kernel[z] = ffma_kernel(z == 0 ? stacked : rows1, a.c.d);
  } else {
    kernel[0] = stacked > 128 ? SharedKernel::kTreeTwo : stacked > kDecodeRows ? SharedKernel::kTreeOne
                                                                              : SharedKernel::kDecode;
    kernel[1] = rows1 > kDecodeRows ? kernel[0] : SharedKernel::kDecode;
  }
  for (int z = 0; z < 2; ++z)
    shape[z] = kernel[z] == SharedKernel::kDecode                                            ? decode_shape(k8)
               : kernel[z] == SharedKernel::kTreeOne || kernel[z] == SharedKernel::kTreeTwo
                   ? tree_shape(a.c.d, kernel[z] == SharedKernel::kTreeTwo)
                   : ffma_shape(kernel[z]);
  // Nothing to gain where a unit has no room for a second sequence's rows, or
  // where all that the table could have in common takes less time to read again
  // than the plan and the join take.
  const int64_t element = held == RA_F32 ? 4 : held == RA_BF16 ? 2 : 1;
  const int64_t again = ((static_cast<int64_t>(B - 1) * a.c.width) << a.c.page_shift) * a.c.heads * 2 * a.c.d * element;
  if (!may_share(B, rows1) || 2 * rows1 > shape[0].rows || rows1 > shape[1].rows || again < kWorthSharing)
    return launch_cache_attention(a, dense, held, s);

  const Room r = room(B, rows1, a.c.heads, a.c.d);
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.ws);
  PlanArgs pl;
  pl.c = a.c;
  pl.shared = shared;
  pl.one_list = kernel[0] == kernel[1];
  pl.lot_rows = shape[0].rows;
  pl.lot_shift = 0;
  while ((1 << pl.lot_shift) < pl.lot_rows) ++pl.lot_shift;
  pl.group = a.Hq / a.c.heads;
  uint8_t* at = ws + r.plan;
  auto take = [&](int64_t bytes) {
    uint8_t* x = at;
    at += round256(bytes);
    return x;
  };
  pl.plan.totals = reinterpret_cast<int64_t*>(take(7 * 8));
  for (int z = 0; z < 2; ++z) {
    const int64_t n = z == 0 ? B + lots_at_most(B, rows1) : B;
    pl.plan.list[z] = reinterpret_cast<Stretch*>(take(n * sizeof(Stretch)));
    pl.tile_shift[z] = 0;
    while ((1 << pl.tile_shift[z]) < shape[z].tile) ++pl.tile_shift[z];
    pl.lead[z] = shape[z].lead;
    pl.ctas[z] = shape[z].ctas;
  }
  pl.plan.places = reinterpret_cast<Place*>(take(B * sizeof(Place)));
  pl.plan.rows_of = reinterpret_cast<int32_t*>(take(stacked * 4));
  const int page = 1 << a.c.page_shift;
  pl.granule = page > kTile ? page : kTile;
  // fewer warps are quicker, where they do not have many rows each
  const int64_t want = B > stacked / 4 ? B : stacked / 4;
  const int threads = want < kPlanThreads ? static_cast<int>((want + 31) / 32 * 32) : kPlanThreads;
  const int smem = B * 32 + 16;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(shared_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kPlanSequences * 32 + 16);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  shared_plan_kernel<<<1, threads, smem, s>>>(pl);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  JoinArgs j;
  j.a = a;
  j.places = pl.plan.places;
  j.first_own = pl.plan.totals + 6;
  j.all_rows = static_cast<int64_t>(B) * a.c.heads * rows1;
  j.rows1 = static_cast<int32_t>(rows1);
  j.lot_rows = pl.lot_rows;
  SharedAttnArgs g;
  static_cast<CacheAttnArgs&>(g) = a;
  static_cast<PagedArgs&>(g.stretches) = a.c;
  g.rows_of = pl.plan.rows_of;
  g.all_rows = j.all_rows;
  g.rows1 = j.rows1;
  for (int z = 0; z < 2; ++z) {
    g.whole_o[z] = reinterpret_cast<float*>(ws + r.whole[z]);
    g.whole_ml[z] = g.whole_o[z] + round256(j.all_rows * a.c.d * 4) / 4;
  }
  for (int z = 0; z < 2; ++z) {
    const int l = pl.one_list ? 0 : z;  // the list, and the launch, of this side
    g.ws = reinterpret_cast<float*>(ws + r.parts[l]);
    g.stretches.list = pl.plan.list[l];
    g.stretches.totals = pl.plan.totals + 3 * l;
    g.stretches.lead = pl.lead[l];
    AttnPlan p;
    p.div = Division{a.c.heads, shape[z].tile, shape[z].ctas};
    p.rows = shape[z].rows;
    p.row_tiles = 1;
    if (z == l) {
      if (kernel[z] == SharedKernel::kDecode)
        e = launch_shared_decode(g, p, k8, s);
      else if (kernel[z] == SharedKernel::kTreeOne || kernel[z] == SharedKernel::kTreeTwo)
        e = launch_shared_tree(g, p, k8, s);
      else
        e = launch_shared_ffma(g, p, kernel[z], k8, s);
      if (e != cudaSuccess) return e;
    }
    const int64_t slots = 2ll * p.div.ctas;
    j.side[z] = Side{g.stretches.list,
                     g.stretches.totals + 2,
                     reinterpret_cast<const float2*>(g.ws),
                     reinterpret_cast<const float4*>(g.ws + slots * p.rows * 2),
                     reinterpret_cast<const float2*>(g.whole_ml[z]),
                     reinterpret_cast<const float4*>(g.whole_o[z]),
                     p.rows,
                     p.div.tile,
                     pl.lead[z],
                     shape[z].quads ? 1 : a.c.d / 4,
                     shape[z].quads ? p.rows : 1};
  }
  // Four warps to a row's parts where those of a single group may be many.
  const int64_t items = (j.all_rows + 31) / 32 * (a.c.d / 4 / kQuads);
  const int64_t units = a.c.heads * ((stacked + pl.lot_rows - 1) / pl.lot_rows);
  const bool many = shape[0].ctas > 16 * units;
  if (dense == RA_BF16) return many ? join<__nv_bfloat16, 4>(j, items, s) : join<__nv_bfloat16, 1>(j, items, s);
  return many ? join<float, 4>(j, items, s) : join<float, 1>(j, items, s);
}

}  // namespace ra
