// Verification of drafted tokens against a model's distributions.
//
// At a node with distribution p, drafts x_1, x_2, .. were drawn from q (row of
// the same node), independently of one another.  With r_0 = p, s_0 = 1:
//   x_k stays iff u_k q(x_k) s_{k-1} < r_{k-1}(x_k); else
//   r_k = max(r_{k-1} - s_{k-1} q, 0),  s_k = sum of r_k.
// What stays is distributed as p whatever q is.  Since q is the same for all of
// a node's drafts, r_k = max(p - c q, 0) with c = s_0 + .. + s_{k-1}: nothing
// of a row has to be kept between its passes.  Drafts that were chosen, not
// drawn (no q), count as drawn with probability 1: r_k is p without the refused
// tokens.  The walk ends at a node all of whose drafts are refused; its next
// token is the first i with r(0) + .. + r(i) > u_0 sum r.
//
// Bound by the bytes of the rows at which sequences stop (V of p and of q),
// and for few sequences by the chain decide - sum - search.  A cluster of CTAs
// takes a sequence, each a part of the row; all walk the tree alike from the
// drafts' own probabilities, which are gathered at the start by one thread
// each, and read a row only where they need its sum.
//
// Decisions have to be those of the definition next to a border as well, and a
// border lies in every 1 / V of the unit interval: sums of fp32 would move 1 %
// of them.  FP64 adds at 1/64 of the rate of fp32, which would bound the pass;
// sums are pairs of floats (error-free sums, 2^-45 and better), and 64 bits decide.
//
// Measured (fp32 unless said): 128 sequences of 5 drafts, V = 131072, 41 to 42 us, of
// which 134 MB of rows take 20 at the copy rate and the chain of a single sequence
// some 11; bf16 35 (22 operations an element for the pairs: issue-bound).  One
// sequence, V = 32768, 14.5 us.  32 trees of 32 chosen tokens, V = 100003, bf16, 25:
// a pass over a row for every node of the path that refuses a token (and one more
// wherever the refused had 7/8 of what was summed), each load, cluster barrier and
// decision, one behind the other.  So the sums of all warps go
// to all CTAs ahead of one barrier, the loads of the parts are under way together
// (31 -> 27 us), and code that runs once stays short, since it is loaded as it
// runs: one place that sums a row, the row's ends in a loop (27 -> 25, one sequence
// 16 -> 14.5).

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cstdint>
#include <utility>

#include "ra_internal.h"
#include "ra_serve.h"

namespace ra {
namespace {

namespace cg = cooperative_groups;

constexpr int kMostCtas = 8;  // of a cluster

// h + l.  What an addition leaves goes to l, which so grows by up to half a step of h
// each time and is rounded to its own 24 bits: every few additions the two are put in
// order again, |l| at most half a step of h.  (Without, the sum of a row of 2^26 with
// half of it in one token was off by 2^-37.6; with it, once a piece, by 2^-45.8.)
struct Pair {
  float h, l;
  __device__ double value() const { return static_cast<double>(h) + l; }
  __device__ void order() {
    const float s = __fadd_rn(h, l);
    l = __fsub_rn(l, __fsub_rn(s, h));
    h = s;
  }
  // += (x, e), both without error but for the last places of l
  __device__ void add(float x, float e) {
    const float s = __fadd_rn(h, x);
    const float z = __fsub_rn(s, h);
    const float err = __fadd_rn(__fsub_rn(h, __fsub_rn(s, z)), __fsub_rn(x, z));
    h = s;
    l = __fadd_rn(l, __fadd_rn(err, e));
  }
};

// max(p - c q, 0) as a pair; NaN stays NaN.
__device__ __forceinline__ Pair rest_of(float p, float q, Pair c) {
  const float m = __fmul_rn(c.h, q);
  const float me = __fmaf_rn(c.l, q, __fmaf_rn(c.h, q, -m));
  const float s = __fsub_rn(p, m);
  const float z = __fsub_rn(s, p);
  const float err = __fsub_rn(__fsub_rn(p, __fsub_rn(s, z)), __fadd_rn(m, z));
  const float e = __fsub_rn(err, me);
  return __fadd_rn(s, e) <= 0.f ? Pair{0.f, 0.f} : Pair{s, e};
}

template <typename E>
struct Piece {  // 16 bytes of a row
  static constexpr int kN = 16 / sizeof(E);
  uint4 w;
  __device__ float get(int i) const {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if (sizeof(E) == 4) return __uint_as_float(x[i % 4]);
    return __uint_as_float(i & 1 ? x[(i / 2) % 4] & 0xffff0000u : x[(i / 2) % 4] << 16);
  }
};
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A node's row, in pieces that lie on 16 bytes: element i of the row is place
// i + shift, and places outside the row hold nothing.
template <typename E, bool kDraft>
struct Row {
  const E* p;
  const E* q;
  int64_t V;
  int shift, whole;  // pieces from here on do not end in the row
  Pair c;
  const int32_t* refused;  // tokens that are out (without q)
  int n_refused;

  __device__ int pieces() const { return static_cast<int>((V + shift + Piece<E>::kN - 1) / Piece<E>::kN); }

  __device__ __forceinline__ Piece<E> load(const E* row, int v) const {
    constexpr int kN = Piece<E>::kN;
    if (v >= (shift > 0) && v < whole) {
      Piece<E> x;
      x.w = __ldg(reinterpret_cast<const uint4*>(row - shift) + v);
      return x;
    }
    // an end of the row, the last element first; few instructions rather than fast:
    // this stands wherever a piece is loaded
    const int64_t first = static_cast<int64_t>(v) * kN - shift;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int i = kN - 1; i >= 0; --i) {
      const bool real = first + i >= 0 && first + i < V;
      const uint32_t bits = real ? __float_as_uint(as_float(row[first + i])) : 0u;
      if (sizeof(E) == 4) {
        w[3] = w[2], w[2] = w[1], w[1] = w[0], w[0] = bits;
      } else {
        w[3] = __funnelshift_l(w[2], w[3], 16);
        w[2] = __funnelshift_l(w[1], w[2], 16);
        w[1] = __funnelshift_l(w[0], w[1], 16);
        w[0] = (w[0] << 16) | (bits >> 16);
      }
    }
    return Piece<E>{make_uint4(w[0], w[1], w[2], w[3])};
  }

  // f(i, rest) for the elements of piece v, whose bytes are x and y
  template <typename F>
  __device__ __forceinline__ void each(int v, const Piece<E>& x, const Piece<E>& y, F f) const {
    constexpr int kN = Piece<E>::kN;
    uint32_t out = 0;  // bit i: element i was refused
    if (!kDraft)
      for (int z = 0; z < n_refused; ++z) {
        const int64_t place = static_cast<int64_t>(refused[z]) + shift;  // passes 32 bits in the longest rows
        if (place / kN == v) out |= 1u << (place % kN);
      }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      Pair r{x.get(i), 0.f};
      if (kDraft) r = rest_of(x.get(i), y.get(i), c);
      if (!kDraft && ((out >> i) & 1u)) r = Pair{0.f, 0.f};
      f(i, r);
    }
  }

  // Piece v of the rows, and what it adds to a sum: nothing behind `last`.
  __device__ __forceinline__ void load(int v, int last, Piece<E>& x, Piece<E>& y) const {
    if (v >= last) return;
    x = load(p, v);
    if (kDraft) y = load(q, v);
  }
  __device__ __forceinline__ void add(int v, int last, const Piece<E>& x, const Piece<E>& y, Pair& s) const {
    if (v >= last) return;
    each(v, x, y, [&](int, Pair r) { s.add(r.h, r.l); });
    s.order();
  }
  __device__ __forceinline__ Pair sum(int v, int last, const Piece<E>& x, const Piece<E>& y) const {
    Pair s{0.f, 0.f};
    add(v, last, x, y, s);
    return s;
  }
  __device__ __forceinline__ Pair sum(int v, int last) const {
    Piece<E> x, y;
    load(v, last, x, y);
    return sum(v, last, x, y);
  }
};

// The sum of the lanes' pairs, in every lane.
__device__ __forceinline__ Pair sum_lanes(Pair x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, x.h, o), l = __shfl_xor_sync(0xffffffffu, x.l, o);
    x.add(h, l);
  }
  x.order();
  return x;
}
__device__ __forceinline__ double scan_lanes(double x) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The first of 32 lanes' values with before + part[0] + .. + part[i] > target, or
// the last that is above 0 where rounding leaves none (-1: none is); `before`
// becomes the sum ahead of it.
__device__ __forceinline__ int crossing(double mine, double target, double& before) {
  const double upto = before + scan_lanes(mine);
  const uint32_t some = __ballot_sync(0xffffffffu, mine > 0.0);
  const uint32_t past = __ballot_sync(0xffffffffu, mine > 0.0 && upto > target);
  const int at = past ? __ffs(past) - 1 : 31 - __clz(some);
  before = __shfl_sync(0xffffffffu, upto - mine, max(at, 0));
  return at;
}

// What the walk asks of the block: a row's sum, for the next decision or, at the
// end, for the next token.
struct Ask {
  int node, n_refused;
  Pair c;
  bool last;
};

// A warp takes its pieces of a row in up to kParts parts, whose sums by lanes it
// leaves in shared memory, so that the search goes on inside one of them.
constexpr int kParts = 8;

template <typename E, bool kDraft, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    verify_kernel(const __grid_constant__ VerifyArgs a) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kAhead = 2;  // rounds of loads under way; 4 are no faster
  extern __shared__ int32_t parent[];                        // [T]
  int32_t* tokens = parent + a.T;                            // [T]
  int32_t* refused = tokens + a.T;                           // [T]
  float* us = reinterpret_cast<float*>(refused + a.T);       // [T]
  float* ps = us + a.T;                                      // [T] p of the parent's row at the token
  float* qs = ps + a.T;                                      // [T]
  __shared__ float2 parts[kWarps][kParts][32];
  // Every CTA has the sums of all warps of the cluster, those of one row until it
  // is through with the next.
  __shared__ float2 warp_sums[2][kMostCtas * kWarps];
  __shared__ double row_total;
  __shared__ Ask ask;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ctas = cluster.num_blocks();
  const int b = blockIdx.x / ctas;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int count = max(0, min(a.count ? a.count[b] : a.T, a.T));
  const int64_t row0 = static_cast<int64_t>(b) * a.T;
  int32_t* path = a.path + row0;
  if (count == 0) {
    if (rank == 0) {
      for (int t = threadIdx.x; t < a.T; t += kThreads) path[t] = -1;
      if (threadIdx.x == 0) {
        a.kept[b] = 0;
        a.token[b] = -1;
      }
    }
    return;  // the whole cluster
  }

  auto begun = cluster.barrier_arrive();
  // ---- the drafts and their own probabilities; -1: not a node of the tree
  for (int t = threadIdx.x; t < count; t += kThreads) {
    const int above = a.parent ? a.parent[row0 + t] : t - 1;
    const int64_t x = a.tokens[row0 + t];
    const bool good = t > 0 && above >= 0 && above < t && x >= 0 && x < a.V;
    parent[t] = good ? above : -1;
    tokens[t] = static_cast<int32_t>(good ? x : 0);
    us[t] = a.uniform[row0 + t];
    const int64_t at = (row0 + above) * a.V + x;
    ps[t] = good ? as_float(static_cast<const E*>(a.probs)[at]) : 0.f;
    qs[t] = good && kDraft ? as_float(static_cast<const E*>(a.draft)[at]) : 1.f;
  }
  __syncthreads();
  bool met = false;

  Row<E, kDraft> row;
  row.V = a.V;
  row.refused = refused;
  // The row's sum, and in every CTA the sums of its parts.
  int turn = 0;
  int w0 = 0, w1 = 0, each = 0;  // this warp's pieces; of a part
  auto row_sum = [&](const Ask& x) {
    const int64_t at = (row0 + x.node) * a.V;
    row.p = static_cast<const E*>(a.probs) + at;
    // where none was refused (c = 0) the rest is p: a node without drafts may have no row of q
    row.q = static_cast<const E*>(kDraft && x.c.h != 0.f ? a.draft : a.probs) + at;
    row.shift = static_cast<int>(at % Piece<E>::kN);
    row.whole = static_cast<int>((a.V + row.shift) / Piece<E>::kN);
    row.c = x.c;
    row.n_refused = x.n_refused;
    const int n = row.pieces();
    const int of_warp = (n + ctas * kWarps - 1) / (ctas * kWarps);
    w0 = min(n, (rank * kWarps + warp) * of_warp);
    w1 = min(n, w0 + of_warp);
    each = (of_warp + kParts * 32 - 1) / (kParts * 32) * 32;  // whole rounds of the warp
    // Loads of some rounds of 32 pieces under way together, those of the next part
    // too: a row of 10^5 has a few rounds a warp.
    const int per = each / 32, rounds = (of_warp + 31) / 32;
    Pair all{0.f, 0.f}, part{0.f, 0.f};
    int filled = 0, left = per;
#pragma unroll 1
    for (int r = 0; r < rounds; r += kAhead) {
      Piece<E> p[kAhead], q[kAhead];
      const int v = w0 + r * 32 + lane;
#pragma unroll
      for (int z = 0; z < kAhead; ++z) row.load(v + 32 * z, w1, p[z], q[z]);
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        row.add(v + 32 * z, w1, p[z], q[z], part);
        if (--left == 0) {
          all.add(part.h, part.l);
          all.order();
          if (filled < kParts) parts[warp][filled++][lane] = make_float2(part.h, part.l);
          part = Pair{0.f, 0.f};
          left = per;
        }
      }
    }
    all.add(part.h, part.l);
    for (; filled < kParts; part = Pair{0.f, 0.f}) parts[warp][filled++][lane] = make_float2(part.h, part.l);
    all = sum_lanes(all);
    turn ^= 1;
    if (!met) cluster.barrier_wait(std::move(begun));  // every CTA is there to be written to
    met = true;
    if (lane < ctas) *cluster.map_shared_rank(&warp_sums[turn][rank * kWarps + warp], lane) = make_float2(all.h, all.l);
    cluster.sync();
    if (warp == 0) {
      Pair total{0.f, 0.f};
      for (int i = lane; i < ctas * kWarps; i += 32) total.add(warp_sums[turn][i].x, warp_sums[turn][i].y);
      total = sum_lanes(total);
      if (lane == 0) row_total = total.value();
      __syncwarp();
    }
  };

  // ---- the walk, by the first warp of every CTA alike (64-bit arithmetic is slow:
  // by all warps a decision took 1 us)
  int node = 0, kept = 1, t = 0, n_refused = 0;
  double total = 1.0, scale = 0.0;  // of what is left of the row; c
  // Without q a refusal only takes its token out, so that a sum serves for the next
  // one too: what it was when it was taken (< 0: not yet) and what has gone from it
  // since.  The difference stands while it is at least kKept of the sum, of which it
  // then keeps all but three bits of the accuracy; where less is left (as of a row
  // with most of its weight on the refused) the row is summed again without them.
  constexpr double kKept = 0.125;
  double whole = -1.0, gone = 0.0;
  bool known = true, summing = false;
  if (rank == 0 && threadIdx.x == 0) path[0] = 0;
  bool walking = true, nothing = false;
  while (true) {
    if (walking && warp == 0) {
      if (summing) {
        whole = total = row_total;
        gone = 0.0;
        known = true;
      }
      while (true) {
        // the next draft below `node`; one that waited for a sum is still at t
        if (!summing) {
          int found = count;
          for (int t0 = t + 1; t0 < count; t0 += 32) {
            const uint32_t here = __ballot_sync(0xffffffffu, t0 + lane < count && parent[t0 + lane] == node);
            if (here) {
              found = t0 + __ffs(here) - 1;
              break;
            }
          }
          t = found;
        }
        summing = false;
        if (t >= count) break;
        if (!known && !kDraft && whole >= 0.0) {
          total = whole - gone;
          known = total >= kKept * whole;
        }
        if (!known) {
          summing = true;
          break;
        }
        const double p = ps[t], q = qs[t];
        double rest = p;
        bool again = false;  // a token that was refused before
        if (kDraft) {
          rest = fmax(p - scale * q, 0.0);
        } else {
          for (int i = 0; i < n_refused; ++i) again = again || refused[i] == tokens[t];
          if (again) rest = 0.0;
        }
        if (us[t] * q * total < rest) {
          if (rank == 0 && lane == 0) path[kept] = t;
          ++kept;
          node = t;
          n_refused = 0;
          total = 1.0;
          scale = gone = 0.0;
          whole = -1.0;
          known = true;
          continue;
        }
        known = false;
        if (kDraft) {
          scale += total;
        } else if (!again) {
          if (lane == 0) refused[n_refused] = tokens[t];
          __syncwarp();
          ++n_refused;
          gone += p;
        }
      }
      if (lane == 0) {
        const float h = static_cast<float>(scale);
        ask = Ask{node, n_refused, Pair{h, static_cast<float>(scale - h)}, !summing};
      }
    }
    __syncthreads();
    Ask x = ask;
    if (nothing) {  // is left: p itself
      x.n_refused = 0;
      x.c = Pair{0.f, 0.f};
    }
    row_sum(x);
    if (!x.last) continue;
    __syncthreads();
    if (nothing || !(row_total <= 0.0)) break;  // (a NaN is no row without a rest)
    nothing = true;
    walking = false;
  }

  // ---- the next token
  const double all = row_total;
  const bool some = all > 0.0 && all < INFINITY;
  if (rank == 0 && warp == 0) {
    for (int i = kept + lane; i < a.T; i += 32) path[i] = -1;
    if (lane == 0) {
      a.kept[b] = kept;
      if (!some) a.token[b] = -1;
    }
  }
  if (some) {
    // warp, part, piece, element: the first warp finds the warp
    __shared__ int found_warp;
    __shared__ double found_before;
    const double target = us[0] * all;
    if (warp == 0) {
      // a lane has the sums of some neighbouring warps
      const int n = ctas * kWarps, of_lane = (n + 31) / 32;
      auto sum_of = [&](int w) { return w < n ? static_cast<double>(warp_sums[turn][w].x) + warp_sums[turn][w].y : 0.0; };
      double before = 0.0, mine = 0.0;
      for (int i = 0; i < of_lane; ++i) mine += sum_of(lane * of_lane + i);
      int found = max(crossing(mine, target, before), 0) * of_lane;
      if (of_lane > 1) found += max(crossing(lane < of_lane ? sum_of(found + lane) : 0.0, target, before), 0);
      if (lane == 0) found_before = before;
      if (lane == 0) found_warp = found - rank * kWarps;
    }
    __syncthreads();
    if (found_warp == warp) {
      double before = found_before;
      double mine = 0.0;  // a lane's: of a part
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const double sum = sum_lanes(Pair{parts[warp][i][lane].x, parts[warp][i][lane].y}).value();
        if (lane == i) mine = sum;
      }
      const int part = max(crossing(mine, target, before), 0);
      const int r0 = min(w1, w0 + part * each), r1 = min(w1, r0 + each);
      // its pieces, 32 at a time, up to those that pass the target
      int v0 = r0;
      double sofar = before, piece = 0.0;  // this lane's of the 32 from v0 on
      for (int i = r0; i < r1; i += 32) {
        const Pair here = row.sum(i + lane, r1);
        const double sum = sum_lanes(here).value();
        if (sum > 0.0) {
          v0 = i;
          before = sofar;
          piece = here.value();
          if (sofar + sum > target) break;
        }
        sofar += sum;
      }
      const int at = crossing(piece, target, before);
      if (at >= 0 && lane == at) {
        const int v = v0 + at;
        const Piece<E> x = row.load(row.p, v), y = row.load(row.q, v);
        int64_t found = -1;
        bool past = false;
        Pair sum{0.f, 0.f};
        row.each(v, x, y, [&](int i, Pair r) {
          if (!past && r.h + r.l > 0.f) {
            found = static_cast<int64_t>(v) * Piece<E>::kN - row.shift + i;
            sum.add(r.h, r.l);
            past = before + sum.value() > target;
          }
        });
        a.token[b] = found;
      }
    }
  }
}

template <typename E, bool kDraft, int kThreads>
cudaError_t launch_k(const VerifyArgs& a, int ctas, cudaStream_t s) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.T) * 24;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(verify_kernel<E, kDraft, kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kVerifyNodes * 24);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  return cudaLaunchKernelEx(&cfg, verify_kernel<E, kDraft, kThreads>, a);
}

template <typename E, bool kDraft>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t s) {
  // All clusters at once on the SMs, 1024 threads on each: few sequences take
  // CTAs of more threads, many of fewer (which spread more evenly over the SMs),
  // and only then fewer CTAs.  (V = 131072, fp32: 64 sequences 27 us with 256
  // threads, 31 with 128; 128 sequences 40 with 128, 41 with 4 CTAs of 512; 512 of
  // 32768 41 and 49.)
  const int64_t held = static_cast<int64_t>(device_sm_count()) * 1024;
  int ctas = kMostCtas;
  if (static_cast<int64_t>(a.B) * ctas * 512 <= held) return launch_k<E, kDraft, 512>(a, ctas, s);
  if (static_cast<int64_t>(a.B) * ctas * 256 <= held) return launch_k<E, kDraft, 256>(a, ctas, s);
  while (ctas > 1 && static_cast<int64_t>(a.B) * ctas * 128 > held) ctas /= 2;
  return launch_k<E, kDraft, 128>(a, ctas, s);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, bool bf16, cudaStream_t s) {
  if (bf16) return a.draft ? launch_t<__nv_bfloat16, true>(a, s) : launch_t<__nv_bfloat16, false>(a, s);
  return a.draft ? launch_t<float, true>(a, s) : launch_t<float, false>(a, s);
}

}  // namespace ra
