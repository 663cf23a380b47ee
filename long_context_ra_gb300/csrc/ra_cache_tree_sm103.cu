// Attention over the paged cache for many query rows per key head (trees of
// drafts, chunks of a prompt): bf16 queries, bf16 or 8-bit cache, tcgen05.
//
// The g x T query rows of a key head are one operand: a unit is up to two
// 128-row tiles of them, and every key tile that is brought in feeds all.
// One persistent CTA per SM walks its run of key tiles (ra_paged.cuh).
//
//   S = Q K^T        tcgen05.mma, bf16 -> fp32 in TMEM
//   p = 2^(s - m)    softmax warps, thread = row, P (bf16) over S in TMEM
//   O += P V         tcgen05.mma
//
// Two streams keep the tensor cores and the exponentials busy together.
// With two query tiles (kTwo) a stream is a query tile and both share the key
// tile; with one, a stream is every other key tile, with a state of its own,
// and the two states are joined at the end of the unit.
//
// Warp roles (512 threads, 128 registers each at launch):
//   warps 0-3, 4-7   softmax of stream 0, 1              (160 registers)
//   warp  8          TMEM allocator, MMA issuer; 9-11 idle (64)
//   warps 12-15      producers                            (128)
// 2 x 128 x 160 + 128 x 64 + 128 x 128 = 65536.
//
// A page may be as short as 8 rows, end inside a tile, or be missing, so the
// producers place the rows themselves: 8 threads own 8 neighbouring rows (one
// page) and write 16-byte pieces where the 128-byte swizzle puts them, zeros
// for rows that do not exist.  bf16 rows go straight to the operand stages
// with cp.async.  8-bit rows go through a raw ring (each thread converts the
// pieces that it loaded itself, so nothing is waited for between threads) and
// become bf16 with the row's scale inside: code * 2^e has 4 significant bits,
// so it is exact in bf16 for values above 2^-126, and neither the scores nor
// the probabilities need to know the scale.
//
// Unseen drafts: their scores are -inf, so p = 0; value rows of tiles with
// drafts are looked through for elements that are not finite.  Those become 0
// in the operand, and a unit that met one adds them at its end, row by row,
// to the queries that see them.
//
// Every wait is bounded, as in the forward kernel.

#include "ra_cache_attn.cuh"
#include "sm103_pipeline.cuh"
#include "sm103_ptx.cuh"

namespace ra {
namespace {

using namespace ptx;
using namespace sm103;

constexpr int kThreads = 512;
constexpr uint32_t kRegsSoftmax = 160, kRegsMma = 64, kRegsLoad = 128;
static_assert(kRegsLoad == 128 && 256 * kRegsSoftmax + 128 * kRegsMma + 128 * kRegsLoad == kThreads * 128,
              "register split must equal the launch's register total");
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 12;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kFastSumBound = 256.0f;  // 2^kRescaleLog2: see the forward kernel

template <bool k8, int D, bool kTwo>
struct Layout {
  static constexpr int kBox = 128 * 128;  // 128 rows x 128 bytes (64 bf16)
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kRawTile = k8 ? 128 * D : 0;
  static constexpr int kStages = D == 128 ? (k8 ? 3 : 5) : (k8 ? 5 : 8);
  static constexpr int kRawStages = 4;
  static constexpr int kLag = k8 ? kRawStages - 1 : 2;  // items in flight
  // the second query tile, or the exchange of the two streams' states:
  // [128][33] floats and [128][2]
  static constexpr int kSecond = kTwo ? kTile : 18 * 1024;
  static constexpr int kQ0 = 0;
  static constexpr int kQ1 = kTile;
  static constexpr int kKV = kTile + kSecond;
  static constexpr int kRaw = kKV + kStages * kTile;
  static constexpr int kRawExp = kRaw + (k8 ? kRawStages * kRawTile : 0);
  static constexpr int kBar = kRawExp + (k8 ? kRawStages * 128 : 0);
  static constexpr int kNumBars = 2 + 2 * kStages + 9;
  static constexpr int kMisc = (kBar + kNumBars * 8 + 15) / 16 * 16;  // TMEM base, abort flag
  static constexpr int kPoison = kMisc + 16;                          // [8]
  static constexpr int kLeftOut = kPoison + 32;                       // [8][16] bytes
  static constexpr int kDivision = kLeftOut + 128;
  // walks of the 8 softmax warps: in shared memory, not in registers
  static constexpr int kWalks = (kDivision + static_cast<int>(sizeof(DivisionShared)) + 15) / 16 * 16;
  static constexpr int kBytes = kWalks + 8 * static_cast<int>(sizeof(UnitWalk));
  static constexpr int kSmem = kBytes + 1024;  // slack for 1024-byte alignment
  static_assert(kSmem <= 232448, "shared memory budget");
};

template <int kStages>
struct Bars {
  uint32_t base;
  __device__ uint32_t q_full() const { return base; }
  __device__ uint32_t q_empty() const { return base + 8; }
  __device__ uint32_t kv_full(int s) const { return base + 8 * (2 + s); }
  __device__ uint32_t kv_empty(int s) const { return base + 8 * (2 + kStages + s); }
  __device__ uint32_t s_full(int t) const { return base + 8 * (2 + 2 * kStages + t); }
  __device__ uint32_t p_full(int t) const { return base + 8 * (4 + 2 * kStages + t); }
  __device__ uint32_t o_full(int t) const { return base + 8 * (6 + 2 * kStages + t); }
  __device__ uint32_t x_full() const { return base + 8 * (8 + 2 * kStages); }
  __device__ uint32_t x_empty() const { return base + 8 * (9 + 2 * kStages); }
  __device__ uint32_t drain() const { return base + 8 * (10 + 2 * kStages); }
};

// Position in a ring of stages.
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  template <int kStages>
  __device__ void step() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Item x of a unit of n key tiles, in the order in which the MMA thread
// takes them: which tile, K or V.  Two query tiles: K0 V0 K1 V1 ...; one:
// K0 K1 V0 K2 V1 ... (two key tiles under way).
template <bool kTwo>
__device__ __forceinline__ void item(int64_t x, int64_t n, int64_t& tile, bool& v) {
  if (kTwo) {
    tile = x >> 1;
    v = x & 1;
  } else if (x == 0) {
    tile = 0;
    v = false;
  } else if (x == 2 * n - 1) {
    tile = n - 1;
    v = true;
  } else {
    v = !(x & 1);
    tile = v ? x / 2 - 1 : (x + 1) / 2;
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
template <int bytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src),
               "r"(real ? bytes : 0), "n"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(at));
  return x;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Halves that are not finite bf16 values, as 0xffff masks.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return ((x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// Two e4m3 values in the high bytes of the halves of x (low bytes zero) times
// the powers of two in `up` and `up2`: sign and 7 bits moved to where bf16
// has them mean value * 2^-120, so up = 2^(120 + e).  A NaN code would come
// out as 480 and is put back.
__device__ __forceinline__ uint32_t widen(uint32_t x, uint32_t up, uint32_t up2, bool twice) {
  uint32_t m = mul_bf16x2((x >> 4) & 0x07f007f0u, up);
  if (twice) m = mul_bf16x2(m, up2);
  m |= ((x & 0x7f00u) == 0x7f00u ? 0x7fffu : 0u) |
       ((x & 0x7f000000u) == 0x7f000000u ? 0x7fff0000u : 0u);
  return m | (x & 0x80008000u);
}

template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint64_t dq, uint64_t dk) {
  constexpr uint32_t idesc = idesc_bf16_f32(kBM, kBN, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = desc_step((kk / 4) * (kBM * 128) + (kk % 4) * 32);
    mma_bf16_ss(d_tmem, dq + off, dk + off, idesc, kk > 0 ? 1u : 0u);
  }
}

template <int D>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t dv,
                                         uint32_t accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(kBM, D, true);
  mma_bf16_ts(d_tmem, p_tmem, dv, idesc, accumulate);
#pragma unroll
  for (int kk = 1; kk < kBN / 16; ++kk)
    mma_bf16_ts(d_tmem, p_tmem + kk * 8, dv + desc_step(kk * 16 * 128), idesc, 1u);
}

// 32 scores of the row, those not in `seen` at -inf.
__device__ __forceinline__ void apply_mask(uint32_t (&s)[32], uint32_t seen) {
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!((seen >> x) & 1u)) s[x] = __float_as_uint(-INFINITY);
}

// f(q, scores of columns 32 q .. 32 q + 31) for the row's 128 scores; the
// next quarter is on its way from TMEM while one is worked on.
template <typename F>
__device__ __forceinline__ void each_quarter(uint32_t tS, bool masked, const uint32_t (&seen)[4], F f) {
  uint32_t s[2][32];
  tmem_ld32(tS, s[0]);
  tmem_ld_wait();
  reg_fence(s[0], 32);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q < 3) tmem_ld32(tS + 32 * (q + 1), s[(q + 1) & 1]);
    if (masked) apply_mask(s[q & 1], seen[q]);
    f(q, s[q & 1]);
    if (q < 3) {
      tmem_ld_wait();
      reg_fence(s[(q + 1) & 1], 32);
    }
  }
}

// p = 2^(s * scale + neg) as bf16 pairs; returns the row's sum.  The scores
// stay in TMEM until the caller stores p over them.
__device__ __forceinline__ float exp_row(uint32_t tS, bool masked, const uint32_t (&seen)[4],
                                         uint64_t scale2, uint64_t neg2, uint32_t (&pk)[64]) {
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
  each_quarter(tS, masked, seen, [&](int q, uint32_t (&s)[32]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint64_t x = fma_f32x2(
          pack_f32x2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), scale2, neg2);
      float x0, x1;
      unpack_f32x2(x, x0, x1);
      const float p0 = ex2(x0), p1 = ex2(x1);
      acc[j & 3] = add_f32x2(acc[j & 3], pack_f32x2(p0, p1));
      pk[16 * q + j] = pack_bf16x2(p0, p1);
    }
  });
  float r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_f32x2(acc[i], r[2 * i], r[2 * i + 1]);
  return ((r[0] + r[1]) + (r[2] + r[3])) + ((r[4] + r[5]) + (r[6] + r[7]));
}

// What a role needs of the present unit.
struct Unit {
  int head;
  int64_t r0;  // first query row of the unit within its key head
  int64_t q0;  // its row in q, out, lse
  __device__ Unit(const CacheAttnArgs& a, const AttnPlan& p, const UnitWalk& u, int64_t rows) {
    head = u.unit / p.row_tiles;
    r0 = static_cast<int64_t>(u.unit % p.row_tiles) * p.rows;
    q0 = (static_cast<int64_t>(u.b) * a.c.heads + head) * rows + r0;
  }
};

template <bool k8, int D, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
    cache_tree_kernel(const __grid_constant__ CacheAttnArgs a, const __grid_constant__ AttnPlan p) {
  using L = Layout<k8, D, kTwo>;
  constexpr int kS = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const Bars<kS> bars{base + L::kBar};
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(gbase + L::kMisc);
  const Abort ab{tmem_holder + 1, a.c.status, a.wait_limit > 0 ? a.wait_limit : kWaitLimit};
  volatile uint32_t* poison = reinterpret_cast<volatile uint32_t*>(gbase + L::kPoison);
  DivisionShared& sh = *reinterpret_cast<DivisionShared*>(gbase + L::kDivision);
  const PagedArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t rows = head_rows(a);

  // ---- set-up
  if (threadIdx.x == 0) {
    mbar_init(bars.q_full(), 128);
    mbar_init(bars.q_empty(), 1);
    for (int s = 0; s < kS; ++s) {
      mbar_init(bars.kv_full(s), 128);
      mbar_init(bars.kv_empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bars.s_full(t), 1);
      mbar_init(bars.p_full(t), 128);
      mbar_init(bars.o_full(t), 1);
    }
    mbar_init(bars.x_full(), 128);
    mbar_init(bars.x_empty(), 128);
    mbar_init(bars.drain(), 1);
    *ab.flag = 0u;
    for (int i = 0; i < 8; ++i) poison[i] = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(base + L::kMisc, kTmemCols);
    tmem_relinquish();
  }
  const int64_t run = division_start(c, p.div, blockIdx.x, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp >= kLoadWarp) {
    // ================= producers =================
    // keeps the registers it was launched with
    const int tid = threadIdx.x - kLoadWarp * 32;
    const int grp = tid / 8, pc = tid % 8;  // rows 8 grp .. 8 grp + 7
    UnitWalk iw, pw;                         // items issued; items handed over
    iw.start(c, p.div, sh, run);
    pw = iw;
    int64_t ix = 0, px = 0;
    int iunit = 0, punit = 0;
    int ktiles = 0;  // K tiles issued, for the left-out ring
    Ring ir, pr;     // operand stages
    int iraw = 0, praw = 0;
    bool ok = static_cast<int64_t>(blockIdx.x) != a.stall_cta;
    const uint8_t* cache_k = static_cast<const uint8_t*>(c.k);
    const uint8_t* cache_v = static_cast<const uint8_t*>(c.v);
    for (int64_t i = 0; ok && !pw.done(); ++i) {
      __syncwarp();  // every lane has read the exponents whose place is refilled now
      // ---- issue one item
      if (!iw.done()) {
        const int64_t n = iw.last - iw.first;
        int64_t tile;
        bool v;
        item<kTwo>(ix, n, tile, v);
        const int64_t pos = (iw.first + tile) * kBN + 8 * grp;
        const int64_t keys = iw.seq.keys();
        int page = -1;
        if (pos < keys) {
          const int64_t col = pos >> c.page_shift;
          if (col < c.width) page = __ldg(c.table + static_cast<int64_t>(iw.b) * c.width + col);
          if (page < 0 || page >= c.pages) {
            page = -1;
            if (pc == 0) flag_page(c.status);
          }
        }
        const int head = iw.unit / p.row_tiles;
        const int64_t row = ((static_cast<int64_t>(page) * c.heads + head) << c.page_shift) +
                            (pos & ((int64_t{1} << c.page_shift) - 1));
        if (!v) {  // which 8-key groups are not in the cache
          if (pc == 0) gbase[L::kLeftOut + (ktiles & 7) * 16 + grp] = pos < keys && page < 0;
          ++ktiles;
        }
        const uint8_t* src = v ? cache_v : cache_k;
        const int nrows = page < 0 ? 0 : static_cast<int>(min(keys - pos, int64_t{8}));
        if (k8) {
          constexpr int kPieces = D / 16;  // of a row
          const uint32_t dst = base + L::kRaw + iraw * L::kRawTile + tid * 16;
          const int r0 = kPieces == 8 ? 0 : (pc / 4) * 4;
          const int cc = kPieces == 8 ? pc : pc % 4;
#pragma unroll
          for (int x = 0; x < kPieces; ++x) {
            const bool real = r0 + x < nrows;
            cp_async16(dst + x * 2048, real ? src + (row + r0 + x) * D + cc * 16 : a.q, real);
          }
          if (pc == 0)
            cp_async_small<8>(base + L::kRawExp + iraw * 128 + grp * 8,
                              nrows > 0 ? static_cast<const void*>((v ? c.ve : c.ke) + row) : a.q,
                              nrows > 0);
          iraw = iraw + 1 == L::kRawStages ? 0 : iraw + 1;
        } else {
          if (!wait_warp(bars.kv_empty(ir.stage), ir.phase ^ 1u, ab)) {
            ok = false;
            break;
          }
          const uint32_t dst = base + L::kKV + ir.stage * L::kTile + grp * 1024;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
#pragma unroll
            for (int b = 0; b < D / 64; ++b) {
              const bool real = x < nrows;
              cp_async16(dst + b * L::kBox + x * 128 + ((pc ^ x) << 4),
                         real ? src + (row + x) * (2 * D) + b * 128 + pc * 16 : a.q, real);
            }
          }
          ir.step<kS>();
        }
        if (++ix == 2 * n) {
          ix = 0;
          ++iunit;
          iw.next(c, p.div);
        }
      }
      cp_commit();
      if (i < L::kLag) continue;

      // ---- hand over the item issued kLag before
      const int64_t n = pw.last - pw.first;
      int64_t tile;
      bool v;
      item<kTwo>(px, n, tile, v);
      if (px == 0) {
        // the unit's queries, ahead of its first key tile
        const Unit un(a, p, pw, rows);
        if (!wait_warp(bars.q_empty(), (punit & 1) ^ 1u, ab)) {
          ok = false;
          break;
        }
        const int qt = kTwo && un.r0 + 128 < rows ? 2 : 1;
        for (int t = 0; t < qt; ++t) {
          const uint32_t dst = base + (t ? L::kQ1 : L::kQ0) + grp * 1024;
          const uint8_t* src = static_cast<const uint8_t*>(a.q) + (un.q0 + t * 128 + 8 * grp) * (2 * D);
          const int64_t left = rows - un.r0 - t * 128 - 8 * grp;
#pragma unroll
          for (int b = 0; b < D / 64; ++b) {
            uint4 q[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
              q[x] = x < left ? *reinterpret_cast<const uint4*>(src + x * 2 * D + b * 128 + pc * 16)
                              : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              st_shared_v4(dst + b * L::kBox + x * 128 + ((pc ^ x) << 4), q[x].x, q[x].y, q[x].z, q[x].w);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bars.q_full());
      }
      const bool border = (pw.first + tile + 1) * kBN > pw.seq.len;
      cp_wait<L::kLag>();
      bool bad = false;
      if (k8) {
        __syncwarp();  // the exponents were loaded by one thread of each group
        if (!wait_warp(bars.kv_empty(pr.stage), pr.phase ^ 1u, ab)) {
          ok = false;
          break;
        }
        constexpr int kPieces = D / 16;
        const uint32_t src = base + L::kRaw + praw * L::kRawTile + tid * 16;
        const uint8_t* ex = gbase + L::kRawExp + praw * 128 + grp * 8;
        const uint32_t dst = base + L::kKV + pr.stage * L::kTile + grp * 1024;
        const int r0 = kPieces == 8 ? 0 : (pc / 4) * 4;
        const int cc = kPieces == 8 ? pc : pc % 4;
        const int box = cc / 4;
        // the two 16-byte halves are written in another order by half of the
        // lanes, so that a row's eight writes meet no bank twice
        const int odd = kPieces == 8 ? box : (pc / 4);
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
          const uint4 w4 = lds128(src + x * 2048);
          const int e = ex[r0 + x];
          const int f1 = min(e + 120, 254);
          const uint32_t up = static_cast<uint32_t>(f1 << 7) * 0x10001u;
          const uint32_t up2 = static_cast<uint32_t>((e + 120 - f1 + 127) << 7) * 0x10001u;
          const bool twice = e > 134;
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          uint32_t o[8];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            o[2 * z] = widen(__byte_perm(w[z], 0u, 0x1404), up, up2, twice);
            o[2 * z + 1] = widen(__byte_perm(w[z], 0u, 0x3424), up, up2, twice);
          }
          if (v && border) {
#pragma unroll
            for (int z = 0; z < 8; ++z) {
              const uint32_t nf = not_finite(o[z]);
              bad = bad || nf;
              o[z] &= ~nf;
            }
          }
          const int r = r0 + x, ch = 2 * (cc % 4);
          const uint32_t at = dst + box * L::kBox + r * 128;
          const uint32_t first = at + (((ch + odd) ^ r) << 4), second = at + (((ch + 1 - odd) ^ r) << 4);
          st_shared_v4(first, odd ? o[4] : o[0], odd ? o[5] : o[1], odd ? o[6] : o[2], odd ? o[7] : o[3]);
          st_shared_v4(second, odd ? o[0] : o[4], odd ? o[1] : o[5], odd ? o[2] : o[6], odd ? o[3] : o[7]);
        }
        praw = praw + 1 == L::kRawStages ? 0 : praw + 1;
      } else if (v && border) {
        const uint32_t dst = base + L::kKV + pr.stage * L::kTile + grp * 1024;
#pragma unroll 1
        for (int x = 0; x < 8 * (D / 64); ++x) {
          const uint32_t at = dst + (x / 8) * L::kBox + (x % 8) * 128 + ((pc ^ (x % 8)) << 4);
          const uint4 w = lds128(at);
          const uint32_t n0 = not_finite(w.x), n1 = not_finite(w.y), n2 = not_finite(w.z),
                         n3 = not_finite(w.w);
          if (n0 | n1 | n2 | n3) {
            bad = true;
            st_shared_v4(at, w.x & ~n0, w.y & ~n1, w.z & ~n2, w.w & ~n3);
          }
        }
      }
      if (bad) poison[punit & 7] = static_cast<uint32_t>(punit) + 1u;
      fence_proxy_async_smem();
      mbar_arrive(bars.kv_full(pr.stage));
      pr.step<kS>();
      if (++px == 2 * n) {
        px = 0;
        ++punit;
        pw.next(c, p.div);
      }
    }
    cp_wait<0>();
  } else if (warp >= kMmaWarp) {
    // ================= MMA issuer =================
    setmaxnreg_dec<kRegsMma>();
    if (warp == kMmaWarp && lane == 0) {
      const uint64_t dQ0 = desc_sw128(base + L::kQ0, 16, 1024);
      const uint64_t dQ1 = desc_sw128(base + L::kQ1, 16, 1024);
      const uint64_t dK = desc_sw128(base + L::kKV, 16, 1024);
      const uint64_t dV = desc_sw128(base + L::kKV, L::kBox, 1024);
      const uint32_t tS0 = tmem, tS1 = tmem + 128, tO0 = tmem + 256, tO1 = tmem + 256 + D;
      Ring r;
      uint32_t unit = 0, np0 = 0, np1 = 0;  // units; P tiles taken per stream
      bool ok = true, any = false;
      UnitWalk u;
      // wait for the next stage of the ring: its index, or -1
      auto take = [&]() {
        if (!wait1(bars.kv_full(r.stage), r.phase, ab)) return -1;
        const int s = r.stage;
        r.step<kS>();
        tc_fence_after();
        return s;
      };
      for (u.start(c, p.div, sh, run); ok && !u.done(); u.next(c, p.div), ++unit) {
        const int n = static_cast<int>(u.last - u.first);
        ok = wait1(bars.q_full(), unit & 1u, ab);
        if (!ok) break;
        any = true;
        int sk = take();
        if (sk < 0) {
          ok = false;
          break;
        }
        if (kTwo) {
          const Unit un(a, p, u, rows);
          const bool two = un.r0 + 128 < rows;
          uint64_t dk = dK + desc_step(sk * L::kTile);
          issue_qk<D>(tS0, dQ0, dk);
          mma_commit(bars.s_full(0));
          if (two) {
            issue_qk<D>(tS1, dQ1, dk);
            mma_commit(bars.s_full(1));
          }
          mma_commit(bars.kv_empty(sk));
          for (int it = 0; it < n; ++it) {
            const int sv = take();
            if (sv < 0 || !wait1(bars.p_full(0), np0++ & 1u, ab)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t dv = dV + desc_step(sv * L::kTile);
            issue_pv<D>(tO0, tS0, dv, it > 0);
            const bool more = it + 1 < n;
            if (more) {
              sk = take();
              if (sk < 0) {
                ok = false;
                break;
              }
              dk = dK + desc_step(sk * L::kTile);
              issue_qk<D>(tS0, dQ0, dk);
              mma_commit(bars.s_full(0));
            }
            if (two) {
              if (!wait1(bars.p_full(1), np1++ & 1u, ab)) {
                ok = false;
                break;
              }
              tc_fence_after();
              issue_pv<D>(tO1, tS1, dv, it > 0);
            }
            mma_commit(bars.kv_empty(sv));
            if (more) {
              if (two) {
                issue_qk<D>(tS1, dQ1, dk);
                mma_commit(bars.s_full(1));
              }
              mma_commit(bars.kv_empty(sk));
            }
          }
          if (ok) {
            mma_commit(bars.q_empty());
            mma_commit(bars.o_full(0));
            if (two) mma_commit(bars.o_full(1));
          }
        } else {
          issue_qk<D>(tS0, dQ0, dK + desc_step(sk * L::kTile));
          mma_commit(bars.s_full(0));
          mma_commit(bars.kv_empty(sk));
          if (n > 1) {
            sk = take();
            if (sk < 0) {
              ok = false;
              break;
            }
            issue_qk<D>(tS1, dQ0, dK + desc_step(sk * L::kTile));
            mma_commit(bars.s_full(1));
            mma_commit(bars.kv_empty(sk));
          }
          for (int it = 0; it < n; ++it) {
            const int t = it & 1;
            const int sv = take();
            if (sv < 0 || !wait1(bars.p_full(t), (t ? np1++ : np0++) & 1u, ab)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t tS = t ? tS1 : tS0;
            issue_pv<D>(t ? tO1 : tO0, tS, dV + desc_step(sv * L::kTile), it > 1);
            mma_commit(bars.kv_empty(sv));
            if (it + 2 < n) {
              sk = take();
              if (sk < 0) {
                ok = false;
                break;
              }
              issue_qk<D>(tS, dQ0, dK + desc_step(sk * L::kTile));
              mma_commit(bars.s_full(t));
              mma_commit(bars.kv_empty(sk));
            }
          }
          if (ok) {
            mma_commit(bars.q_empty());
            mma_commit(bars.o_full(0));
            if (n > 1) mma_commit(bars.o_full(1));
          }
        }
      }
      if (!ok && any) {
        mma_commit(bars.drain());
        wait_drain(bars.drain(), 0);
      }
    }
  } else {
    // ================= softmax =================
    setmaxnreg_inc<kRegsSoftmax>();
    const int t = warp / 4, wq = warp % 4;
    const int row = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(t * 128);
    const uint32_t tO = tmem + lane_off + 256u + static_cast<uint32_t>(t * D);
    const uint64_t scale2 = pack_f32x2(a.scale_log2, a.scale_log2);
    float* xo = reinterpret_cast<float*>(gbase + L::kQ1);  // [128][33]
    float* xml = xo + 128 * 33;                            // [128][2]
    uint32_t ns = 0, no = 0, unit = 0, xc = 0, kt = 0;     // phases; K tiles before the unit
    bool ok = true;
    UnitWalk& u = reinterpret_cast<UnitWalk*>(gbase + L::kWalks)[warp];
    if (lane == 0) u.start(c, p.div, sh, run);
    __syncwarp();
    while (ok && !u.done()) {
      const int n = static_cast<int>(u.last - u.first);
      // the first tile of this part that holds drafts or the end
      const int border = static_cast<int>(
          min(max(u.seq.len / kBN - u.first, int64_t{0}), static_cast<int64_t>(n)));
      int tok;
      bool active, exists;
      {
        const Unit un(a, p, u, rows);
        active = kTwo ? (t == 0 || un.r0 + 128 < rows) : (t == 0 || n > 1);
        const int64_t lrow = un.r0 + (kTwo ? t * 128 : 0) + row;  // row within the key head
        exists = lrow < rows;
        tok = exists ? static_cast<int>(lrow % c.T) : c.T;
      }
      const bool live = tok < u.seq.cnt;
      const bool warp_live = __any_sync(0xffffffffu, live);
      float m_ref = -INFINITY, l = 0.f;
      if (active) {
        bool o_valid = false;
        for (int it = kTwo ? 0 : t; it < n; it += kTwo ? 1 : 2) {
          if (!wait_warp(bars.s_full(t), ns++ & 1u, ab)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (warp_live) {
            const uint4 left = lds128(base + L::kLeftOut + ((kt + it) & 7u) * 16u);
            const bool masked = it >= border || (left.x | left.y | left.z | left.w);
            uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
            if (masked) {
              const int64_t pos = (u.first + it) * kBN;
              const uint32_t lw[4] = {left.x, left.y, left.z, left.w};
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                seen[w] = 0;
#pragma unroll 1
                for (int x = 0; x < 32; ++x) {
                  const bool out = (lw[w] >> (8 * (x / 8))) & 0xffu;
                  if (!out && sees(a, u.seq, u.b, tok, pos + 32 * w + x)) seen[w] |= 1u << x;
                }
              }
            }
            // As in the forward: exponentials against the present reference
            // first; a row sum of at most 2^kRescaleLog2 rules out that the
            // reference has to move.
            uint32_t pk[64];
            bool redo = true;
            if (__all_sync(0xffffffffu, m_ref != -INFINITY)) {
              const float lt = exp_row(tS, masked, seen, scale2, pack_f32x2(-m_ref, -m_ref), pk);
              if (!__any_sync(0xffffffffu, lt > kFastSumBound)) {
                l += lt;
                redo = false;
              }
            }
            if (redo) {
              float mx = -INFINITY;
              each_quarter(tS, masked, seen, [&](int, uint32_t (&s)[32]) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(s[e]);
#pragma unroll
                for (int j = 4; j < 28; j += 8)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    v[e] = fmax3(v[e], __uint_as_float(s[j + e]), __uint_as_float(s[j + 4 + e]));
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = fmaxf(v[e], __uint_as_float(s[28 + e]));
                mx = fmax3(mx, fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
              });
              const float m_new = mx * a.scale_log2;
              const bool need = m_new > m_ref + kRescaleLog2;
              if (__any_sync(0xffffffffu, need)) {
                const float alpha = need ? ex2(m_ref - m_new) : 1.f;
                if (o_valid) {
#pragma unroll
                  for (int x = 0; x < D; x += 32) {
                    uint32_t r[32];
                    tmem_ld32(tO + x, r);
                    tmem_ld_wait();
                    reg_fence(r, 32);
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                    tmem_st32(tO + x, r);
                  }
                  tmem_st_wait();
                }
                if (need) {
                  l *= alpha;
                  m_ref = m_new;
                }
              }
              // a row that has seen no key yet keeps m_ref = -inf: p = 0, not NaN
              const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
              l += exp_row(tS, masked, seen, scale2, pack_f32x2(neg, neg), pk);
            }
            tmem_st32(tS, pk);
            tmem_st32(tS + 32, pk + 32);
            tmem_st_wait();
          }
          tc_fence_before();
          mbar_arrive(bars.p_full(t));
          o_valid = true;
        }
        if (!ok) break;
        if (!wait_warp(bars.o_full(t), no++ & 1u, ab)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      kt += static_cast<uint32_t>(n);
      if (!live) {
        m_ref = -INFINITY;
        l = 0.f;
      }
      const bool poisoned = poison[unit & 7] == unit + 1u;

      // ---- one query tile: stream 1 hands its state to stream 0
      const bool exchange = !kTwo && n > 1;
      float f0 = 1.f, f1 = 0.f;  // weights of the two streams' sums
      if (exchange && t == 1) {
        if (!wait_warp(bars.x_empty(), (xc & 1u) ^ 1u, ab)) {
          ok = false;
          break;
        }
        xml[2 * row] = m_ref;
        xml[2 * row + 1] = l;
      }
      if (kTwo ? active : true) {
        const Unit un(a, p, u, rows);
        const bool whole = u.whole();
        const int slot = u.slot(blockIdx.x);
        const int local = (kTwo ? t * 128 : 0) + row;
        float inv = 1.f;
        for (int x = 0; x < D; x += 32) {
          uint32_t r[32];
          if (active) {
            tmem_ld32(tO + x, r);
            tmem_ld_wait();
            reg_fence(r, 32);
          }
          if (!kTwo && t == 1) {
            if (!exchange) break;
            if (x > 0 && !wait_warp(bars.x_empty(), (xc & 1u) ^ 1u, ab)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) xo[row * 33 + e] = __uint_as_float(r[e]);
            mbar_arrive(bars.x_full());
            ++xc;
            continue;
          }
          if (exchange) {
            if (!wait_warp(bars.x_full(), xc & 1u, ab)) {
              ok = false;
              break;
            }
            if (x == 0) {
              const float m1 = xml[2 * row], l1 = xml[2 * row + 1];
              const float ms = fmaxf(m_ref, m1);
              f0 = l == 0.f ? 0.f : ex2(m_ref - ms);
              f1 = l1 == 0.f ? 0.f : ex2(m1 - ms);
              l = f0 * l + f1 * l1;
              m_ref = ms;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float y = xo[row * 33 + e];
              float z = f0 == 0.f ? 0.f : f0 * __uint_as_float(r[e]);
              if (f1 != 0.f) z = fmaf(f1, y, z);
              r[e] = __float_as_uint(z);
            }
            mbar_arrive(bars.x_empty());
            ++xc;
          }
          if (x == 0 && whole) inv = l == 0.f ? 0.f : 1.f / l;
          if (l == 0.f) {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0u;
          }
          if (poisoned && live) {
            // elements of the drafts that were left out because they are not finite
            int64_t pos = max(u.first * kBN, u.seq.len);
            const int64_t end = min(u.last * kBN, u.seq.keys());
            for (; pos < end; ++pos) {
              if (!sees(a, u.seq, u.b, tok, pos)) continue;
              const int64_t at = cache_row(c, u.b, pos);
              if (at < 0) continue;
              const int64_t vr = at + (static_cast<int64_t>(un.head) << c.page_shift);
#pragma unroll 1
              for (int e = 0; e < 32; ++e) {
                float y;
                if (k8) {
                  const uint8_t code = static_cast<const uint8_t*>(c.v)[vr * D + x + e];
                  const uint32_t z = widen(static_cast<uint32_t>(code) << 8,
                                           static_cast<uint32_t>(min(c.ve[vr] + 120, 254)) << 7,
                                           static_cast<uint32_t>(c.ve[vr] + 247 - min(c.ve[vr] + 120, 254)) << 7,
                                           c.ve[vr] > 134);
                  y = __uint_as_float(z << 16);
                } else {
                  y = __uint_as_float(static_cast<uint32_t>(
                          static_cast<const uint16_t*>(c.v)[vr * D + x + e]) << 16);
                }
                if (!isfinite(y)) {
#pragma unroll
                  for (int z = 0; z < 32; ++z)
                    if (z == e) r[z] = 0x7fffffffu;
                }
              }
            }
          }
          if (exists) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (un.q0 + local) * D + x);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint4 w;
                w.x = pack_bf16x2(__uint_as_float(r[8 * e + 0]) * inv, __uint_as_float(r[8 * e + 1]) * inv);
                w.y = pack_bf16x2(__uint_as_float(r[8 * e + 2]) * inv, __uint_as_float(r[8 * e + 3]) * inv);
                w.z = pack_bf16x2(__uint_as_float(r[8 * e + 4]) * inv, __uint_as_float(r[8 * e + 5]) * inv);
                w.w = pack_bf16x2(__uint_as_float(r[8 * e + 6]) * inv, __uint_as_float(r[8 * e + 7]) * inv);
                dst[e] = w;
              }
              if (x == 0)
                a.lse[un.q0 + local] = l == 0.f ? -INFINITY : (m_ref + __log2f(l)) * kLn2F;
            } else {
              float4* dst = reinterpret_cast<float4*>(slot_o(a, p, slot) + static_cast<int64_t>(local) * D + x);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                dst[e] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                     __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
              if (x == 0) {
                float* ml = slot_ml(a, p, slot) + 2 * local;
                ml[0] = m_ref;
                ml[1] = l;
              }
            }
          }
        }
        tc_fence_before();
      }
      ++unit;
      __syncwarp();
      if (lane == 0) u.next(c, p.div);
      __syncwarp();
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool k8, int D, bool kTwo>
cudaError_t launch_t(const CacheAttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  using L = Layout<k8, D, kTwo>;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(cache_tree_kernel<k8, D, kTwo>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cache_tree_kernel<k8, D, kTwo><<<p.div.ctas, kThreads, L::kSmem, s>>>(a, p);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_cache_attn_join(a, p, true, s) : e;
}

template <bool k8, int D>
cudaError_t by_rows(const CacheAttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  return p.rows == 256 ? launch_t<k8, D, true>(a, p, s) : launch_t<k8, D, false>(a, p, s);
}

}  // namespace

cudaError_t launch_cache_tree(const CacheAttnArgs& a, bool k8, cudaStream_t s) {
  AttnPlan p;
  const int64_t rows = head_rows(a);
  p.rows = rows > 128 ? 256 : 128;
  p.row_tiles = static_cast<int>((rows + p.rows - 1) / p.rows);
  p.div.units = a.c.heads * p.row_tiles;
  p.div.tile = kBN;
  p.div.ctas = kTreeCtas;
  p.div.min_run = 1;
  if (a.c.d == 128) return k8 ? by_rows<true, 128>(a, p, s) : by_rows<false, 128>(a, p, s);
  return k8 ? by_rows<true, 64>(a, p, s) : by_rows<false, 64>(a, p, s);
}

}  // namespace ra
