// Pages of the cache that several sequences may hold: forks, room for new
// tokens, release, and the copies and moves that follow.
//
// ref[page] counts the rows of tables that hold a page; 0 is free, and there
// is no other list of free pages: a reservation takes the lowest free numbers
// in the order (sequence, column), so the same state gives the same pages
// whatever the order in which threads run, and no state can disagree with
// another.  Counts change by integer atomics, whose order does not matter.
//
// Bound by launches and by chains of loads (times of a call among others of its kind,
// behind one another): a fork reads a row of the table and adds to its pages' counts,
// a block per row, 5 us; a reservation is one block, 6 us for 4 sequences and 9 for 96
// with trees of 32 (who asks; the counts of the pages they hold; a scan over them; the
// free pages, 16 a thread and round); copies and moves go with 16 bytes a lane, four
// or eight of them under way (96 forks, of which 64 copy a page of 2 x 128 KB: 8 us; 192
// sequences' 64 nodes, 12 MB in scattered rows, 8).  96 beams' release, fork, room and
// copy by graph replay 23 us, of which 48 MB take 7 at the copy rate.
// Rounds beyond the first are slow: one block looks at 16384 pages in some 4 us, and
// twice, so a pool whose free pages lie behind 95000 held ones takes 60 us a
// reservation, behind 950000 540.

#include "ra_paged.cuh"

namespace ra {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ int held_columns(const PageTableArgs& a, int b) {
  return max(0, min(a.held[b], a.width));
}
__device__ __forceinline__ int64_t columns_of(const PageTableArgs& a, int64_t tokens) {
  return (tokens + (int64_t{1} << a.page_shift) - 1) >> a.page_shift;
}
__device__ __forceinline__ bool a_page(const PageTableArgs& a, int p) { return p >= 0 && p < a.pages; }

// A block per new row: the source's columns, one holder more for each.
__global__ void __launch_bounds__(kRowThreads)
    pages_fork_kernel(const __grid_constant__ PageTableArgs a, const int32_t* source, int32_t* table_out,
                      int32_t* held_out, int32_t* lens_out) {
  const int i = blockIdx.x;
  const int b = source[i];
  const bool live = b >= 0 && b < a.B && a.lens[b] >= 0;
  int n = 0;
  bool bad = b >= a.B;
  if (live) {
    const int64_t want = columns_of(a, a.lens[b]);
    n = static_cast<int>(min(want, static_cast<int64_t>(held_columns(a, b))));
    bad = n < want;  // a context that is not held
  }
  const int32_t* from = a.table + static_cast<int64_t>(live ? b : 0) * a.width;
  int32_t* to = table_out + static_cast<int64_t>(i) * a.width;
  for (int c = threadIdx.x; c < a.width; c += kRowThreads) {
    int p = -1;
    if (c < n) {
      p = from[c];
      if (a_page(a, p)) {
        atomicAdd(a.ref + p, 1);
      } else {
        p = -1;
        bad = true;
      }
    }
    to[c] = p;
  }
  if (bad) flag_page(a.status);
  if (threadIdx.x == 0) {
    held_out[i] = n;
    lens_out[i] = live ? a.lens[b] : -1;
  }
}

// A block per sequence: the columns behind its tokens are given back.
__global__ void __launch_bounds__(kRowThreads)
    pages_trim_kernel(const __grid_constant__ PageTableArgs a) {
  const int b = blockIdx.x;
  const int held = held_columns(a, b);
  const int64_t want = a.lens && a.lens[b] >= 0 ? columns_of(a, a.lens[b]) : 0;
  const int keep = static_cast<int>(min(want, static_cast<int64_t>(held)));
  int32_t* row = a.table + static_cast<int64_t>(b) * a.width;
  bool bad = false;
  for (int c = keep + threadIdx.x; c < held; c += kRowThreads) {
    const int p = row[c];
    row[c] = -1;
    if (!a_page(a, p)) {
      bad = true;
    } else if (atomicSub(a.ref + p, 1) <= 0) {  // nobody held it: the count stays as it was
      atomicAdd(a.ref + p, 1);
      bad = true;
    }
  }
  if (bad) flag_page(a.status);
  __syncthreads();
  if (threadIdx.x == 0) a.held[b] = keep;
}

// ---------------------------------------------------------------- reserve
// One block, since the pages' numbers depend on every sequence's need.  A
// sequence that writes into a page which others hold as well leaves it for a
// fresh one.  Where all who hold a page ask for room, the last of them may
// keep it: all take one off the count, and where nothing is left of it they
// leave the smallest -(b + 1) in its place, which the one that keeps the page
// finds there.
constexpr int kReserveThreads = 1024;
constexpr int kScan = 16;  // pages a thread looks at in a round

enum : uint8_t { kAsksNothing = 0, kAsks = 1, kLeaves = 2, kKeeps = 3 };

// Inclusive scan of one int per thread; all = the sum.
__device__ __forceinline__ int scan_block(int x, int* warps, int& all) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  int w = warps[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return x + (warp > 0 ? before : 0);
}

// A thread has the sequences tid, tid + 1024, .. and keeps what it has read of
// them: the block spends its time on chains of loads.
constexpr int kEach = kReserveSequences / kReserveThreads;

__global__ void __launch_bounds__(kReserveThreads)
    pages_reserve_kernel(const __grid_constant__ PageTableArgs a, const int32_t* count, int T, int32_t* granted,
                         int32_t* src, int32_t* dst) {
  extern __shared__ int32_t upto[];  // [B] pages wanted up to and with a sequence
  uint8_t* state = reinterpret_cast<uint8_t*>(upto + a.B);
  __shared__ int warps[32];
  const int tid = threadIdx.x;
  const int64_t in_page = (int64_t{1} << a.page_shift) - 1;
  // f(b, i) for this thread's sequences, the i-th of them
  auto mine = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int b = tid + i * kReserveThreads;
      if (i * kReserveThreads >= a.B) break;
      if (b < a.B) f(b, i);
    }
  };
  int len[kEach], tokens[kEach], held[kEach], page[kEach];  // page: of the first new token, where others hold it too
  uint8_t st[kEach];

  // ---- who asks, and for how much
  mine([&](int b, int i) {
    len[i] = a.lens[b];
    tokens[i] = count ? count[b] : T;
    held[i] = held_columns(a, b);
  });
  bool leaving = false;
  mine([&](int b, int i) {
    int need = 0;
    st[i] = kAsksNothing;
    page[i] = -1;
    if (len[i] >= 0 && tokens[i] > T) flag_page(a.status);
    tokens[i] = max(0, min(tokens[i], T));
    if (len[i] >= 0 && tokens[i] > 0) {
      const int64_t last = columns_of(a, static_cast<int64_t>(len[i]) + tokens[i]);
      bool good = last <= a.width && columns_of(a, len[i]) <= held[i];
      if (good) {
        const int32_t* row = a.table + static_cast<int64_t>(b) * a.width;
        const int first = len[i] >> a.page_shift;
        for (int c = first; c < min(static_cast<int64_t>(held[i]), last); ++c) {
          const int p = row[c];
          const int r = a_page(a, p) ? a.ref[p] : 0;
          if (r > 1 && c == first) page[i] = p;
          good = good && r >= 1 && (r == 1 || c == first);
        }
      }
      if (good) {
        st[i] = page[i] >= 0 ? kLeaves : kAsks;
        need = static_cast<int>(max(last - held[i], int64_t{0}));
        leaving = leaving || st[i] == kLeaves;
      } else {
        flag_page(a.status);
      }
    }
    upto[b] = need;
    src[b] = -1;
    dst[b] = -1;
  });
  if (__syncthreads_or(leaving)) {  // (all counts have been read)
    mine([&](int, int i) {
      if (st[i] == kLeaves) atomicSub(a.ref + page[i], 1);
    });
    __syncthreads();
    mine([&](int b, int i) {
      if (st[i] == kLeaves && __ldcg(a.ref + page[i]) <= 0) atomicMin(a.ref + page[i], -(b + 1));
    });
    __syncthreads();
    mine([&](int b, int i) {
      if (st[i] != kLeaves) return;
      if (__ldcg(a.ref + page[i]) == -(b + 1))
        st[i] = kKeeps;
      else
        upto[b] += 1;
    });
    __syncthreads();
    mine([&](int, int i) {
      if (st[i] == kKeeps) a.ref[page[i]] = 1;
    });
  }
  mine([&](int b, int i) { state[b] = st[i]; });
  __syncthreads();

  // ---- upto: an inclusive scan, a run of sequences per thread
  int total;  // below 2^31: B rows of the table
  {
    const int each = (a.B + kReserveThreads - 1) / kReserveThreads;
    const int b0 = min(a.B, tid * each), b1 = min(a.B, b0 + each);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += upto[b];
    int at = scan_block(sum, warps, total) - sum;
    for (int b = b0; b < b1; ++b) {
      at += upto[b];
      upto[b] = at;
    }
  }
  __syncthreads();

  // ---- free pages in rising order, f(page, rank) for those below `total`.  The
  // second walk has the first round's pages still in hand.
  uint32_t first_free = 0;
  int first_rank = 0, first_all = 0;
  auto look = [&](int64_t p0, int& rank, int& all) {
    const int64_t p = p0 + tid * kScan;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kScan; ++i)
      if (p + i < a.pages && __ldcg(a.ref + p + i) == 0) bits |= 1u << i;
    rank = scan_block(__popc(bits), warps, all) - __popc(bits);
    return bits;
  };
  constexpr int64_t kRound = static_cast<int64_t>(kReserveThreads) * kScan;
  bool enough = total == 0;
  if (!enough) {
    first_free = look(0, first_rank, first_all);
    int found = first_all;
    for (int64_t p0 = kRound; p0 < a.pages && found < total; p0 += kRound) {
      int rank, all;
      look(p0, rank, all);
      found += all;
    }
    enough = found >= total;
  }
  if (!enough) {  // all or nothing
    if (tid == 0) flag_page(a.status);
    mine([&](int b, int i) {
      if (st[i] == kLeaves) atomicAdd(a.ref + page[i], 1);
      granted[b] = 0;
    });
    return;
  }
  auto give = [&](int page_number, int rank) {
    int lo = 0, hi = a.B - 1;  // the first sequence with upto > rank
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (upto[mid] > rank)
        hi = mid;
      else
        lo = mid + 1;
    }
    int j = rank - (lo > 0 ? upto[lo - 1] : 0);
    int32_t* row = a.table + static_cast<int64_t>(lo) * a.width;
    a.ref[page_number] = 1;
    if (state[lo] == kLeaves && j-- == 0) {
      const int at = a.lens[lo], first = at >> a.page_shift;
      if (at & in_page) {  // tokens of the context lie in it
        src[lo] = row[first];
        dst[lo] = page_number;
      }
      row[first] = page_number;
      return;
    }
    row[held_columns(a, lo) + j] = page_number;
  };
  int before = 0;
  for (int64_t p0 = 0; p0 < a.pages && before < total; p0 += kRound) {
    int rank = first_rank, all = first_all;
    uint32_t bits = first_free;
    if (p0 > 0) bits = look(p0, rank, all);
    for (rank += before; bits && rank < total; bits &= bits - 1, ++rank)
      give(static_cast<int>(p0 + tid * kScan + __ffs(bits) - 1), rank);
    before += all;
  }
  __syncthreads();  // the columns that were held have been read
  mine([&](int b, int i) {
    const bool asks = st[i] != kAsksNothing;
    granted[b] = asks ? tokens[i] : 0;
    if (asks)
      a.held[b] = static_cast<int32_t>(
          max(static_cast<int64_t>(held[i]), columns_of(a, static_cast<int64_t>(len[i]) + tokens[i])));
  });
}

// ------------------------------------------------------------------- copy
// A page of one side is one piece of memory.  A block moves kCopyBytes of it,
// four 16-byte loads a thread on their way together.
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = kCopyThreads * 16 * 4;

__global__ void __launch_bounds__(kCopyThreads)
    cache_copy_kernel(const __grid_constant__ PagedArgs c, const int32_t* src, const int32_t* dst,
                      int n, int64_t page_bytes, int chunks) {
  const bool v = static_cast<int>(blockIdx.x) >= chunks;
  const int chunk = blockIdx.x - (v ? chunks : 0);
  uint8_t* side = static_cast<uint8_t*>(v ? c.v : c.k);
  const int64_t at = static_cast<int64_t>(chunk) * kCopyBytes + threadIdx.x * 16;
  for (int i = blockIdx.y; i < n; i += gridDim.y) {
    const int64_t from = src[i], to = dst[i];
    if (from < 0 || to < 0) continue;
    if (from >= c.pages || to >= c.pages) {
      if (threadIdx.x == 0 && blockIdx.x == 0) flag_page(c.status);
      continue;
    }
    const uint8_t* s = side + from * page_bytes;
    uint8_t* d = side + to * page_bytes;
    uint4 x[4];
#pragma unroll
    for (int z = 0; z < 4; ++z)
      if (at + z * (kCopyThreads * 16) < page_bytes)
        x[z] = *reinterpret_cast<const uint4*>(s + at + z * (kCopyThreads * 16));
#pragma unroll
    for (int z = 0; z < 4; ++z)
      if (at + z * (kCopyThreads * 16) < page_bytes)
        *reinterpret_cast<uint4*>(d + at + z * (kCopyThreads * 16)) = x[z];
    if (c.ke && chunk == 0) {
      const int64_t rows = static_cast<int64_t>(c.heads) << c.page_shift;  // a multiple of 8
      uint8_t* e = v ? c.ve : c.ke;
      for (int64_t z = threadIdx.x * 8; z < rows; z += kCopyThreads * 8)
        *reinterpret_cast<uint2*>(e + to * rows + z) = *reinterpret_cast<const uint2*>(e + from * rows + z);
    }
  }
}

// ---------------------------------------------------------------- compact
// A thread has one piece (V bytes) of one head's row of K or V and walks over
// the kept tokens.  Since they rise, token j's row moves to a place at or
// before its own, which no later token reads: rows are loaded kAhead at a time
// and stored, in order.
constexpr int kCompactThreads = 128;
constexpr int kCompactTokens = 128;  // looked up at a time

template <typename V>
__global__ void __launch_bounds__(kCompactThreads)
    cache_compact_kernel(const __grid_constant__ PagedArgs c, const int32_t* path, int pieces) {
  constexpr int kAhead = 8;
  __shared__ int64_t from[kCompactTokens], to[kCompactTokens];
  __shared__ int end;
  const int b = blockIdx.x;
  const int64_t len = c.lens[b];
  const int kept = len < 0 ? 0 : max(0, min(c.count[b], c.T));
  if (len >= 0 && c.count[b] > c.T && threadIdx.x == 0) flag_page(c.status);
  const int item = blockIdx.y * kCompactThreads + threadIdx.x;
  const int row = item / pieces, piece = item % pieces;
  const bool live = row < 2 * c.heads;
  const bool v = row >= c.heads;
  V* side = static_cast<V*>(v ? c.v : c.k) + piece;
  uint8_t* exps = v ? c.ve : c.ke;
  const int64_t head = static_cast<int64_t>(v ? row - c.heads : row) << c.page_shift;
  const int32_t* nodes = path + static_cast<int64_t>(b) * c.T;
  for (int j0 = 0; j0 < kept; j0 += kCompactTokens) {
    __syncthreads();
    if (threadIdx.x == 0) end = kCompactTokens;
    __syncthreads();
    const int j = j0 + threadIdx.x;
    if (threadIdx.x < kCompactTokens && j < kept) {
      const int node = nodes[j];
      const int before = j > 0 ? nodes[j - 1] : -1;
      if (node <= before || node >= c.T) {
        atomicMin(&end, static_cast<int>(threadIdx.x));
        flag_page(c.status);
      } else {
        const int64_t f = node == j ? -1 : cache_row(c, b, len + node);
        from[threadIdx.x] = f;
        to[threadIdx.x] = f < 0 ? -1 : cache_row(c, b, len + j);
      }
    }
    __syncthreads();
    const int n = min(end, min(kept - j0, kCompactTokens));
    if (live) {
      for (int i0 = 0; i0 < n; i0 += kAhead) {
        V x[kAhead];
        uint8_t e[kAhead];
#pragma unroll
        for (int z = 0; z < kAhead; ++z) {
          const int i = i0 + z;
          if (i < n && to[i] >= 0) {
            x[z] = side[(from[i] + head) * pieces];
            if (exps && piece == 0) e[z] = exps[from[i] + head];
          }
        }
#pragma unroll
        for (int z = 0; z < kAhead; ++z) {
          const int i = i0 + z;
          if (i < n && to[i] >= 0) {
            side[(to[i] + head) * pieces] = x[z];
            if (exps && piece == 0) exps[to[i] + head] = e[z];
          }
        }
      }
    }
    if (n < kCompactTokens) break;
  }
}

int64_t row_bytes(const PagedArgs& c, ra_dtype held) {
  return static_cast<int64_t>(c.d) * (held == RA_F32 ? 4 : held == RA_BF16 ? 2 : 1);
}

}  // namespace

cudaError_t launch_pages_fork(const PageTableArgs& a, const int32_t* source, int32_t n, int32_t* table_out,
                              int32_t* held_out, int32_t* lens_out, cudaStream_t s) {
  pages_fork_kernel<<<n, kRowThreads, 0, s>>>(a, source, table_out, held_out, lens_out);
  return cudaGetLastError();
}

cudaError_t launch_pages_trim(const PageTableArgs& a, cudaStream_t s) {
  pages_trim_kernel<<<a.B, kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pages_reserve(const PageTableArgs& a, const int32_t* count, int32_t T, int32_t* granted,
                                 int32_t* src, int32_t* dst, cudaStream_t s) {
  static_assert(kReserveSequences * 5 <= 48 * 1024, "shared memory without opt-in");
  pages_reserve_kernel<<<1, kReserveThreads, a.B * 5, s>>>(a, count, T, granted, src, dst);
  return cudaGetLastError();
}

cudaError_t launch_cache_copy(const PagedArgs& c, ra_dtype held, const int32_t* src, const int32_t* dst, int32_t n,
                              cudaStream_t s) {
  const int64_t bytes = (row_bytes(c, held) * c.heads) << c.page_shift;
  const int chunks = static_cast<int>((bytes + kCopyBytes - 1) / kCopyBytes);
  cache_copy_kernel<<<dim3(2 * chunks, n < 65535 ? n : 65535), kCopyThreads, 0, s>>>(c, src, dst, n, bytes, chunks);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const PagedArgs& c, ra_dtype held, const int32_t* path, cudaStream_t s) {
  const int64_t bytes = row_bytes(c, held);
  const bool wide = bytes % 16 == 0;
  const int pieces = static_cast<int>(bytes / (wide ? 16 : 8));
  const dim3 grid(c.B, (2 * c.heads * pieces + kCompactThreads - 1) / kCompactThreads);
  if (wide)
    cache_compact_kernel<uint4><<<grid, kCompactThreads, 0, s>>>(c, path, pieces);
  else
    cache_compact_kernel<uint2><<<grid, kCompactThreads, 0, s>>>(c, path, pieces);
  return cudaGetLastError();
}

}  // namespace ra
