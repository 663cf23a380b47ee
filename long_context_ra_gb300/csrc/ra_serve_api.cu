// C ABI of the calls around the attention: query/key norm with rotation, the
// paged cache and the attention over it.  Every check runs before anything
// is enqueued.

#include <cmath>
#include <cstdint>

#include "ra.h"
#include "ra_internal.h"
#include "ra_serve.h"
#include "ra_trace.h"

namespace ra {
namespace {

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
ra_status launched(cudaError_t e) { return e == cudaSuccess ? RA_OK : RA_ERR_CUDA; }
cudaStream_t cu(ra_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int64_t kMaxTokens = (int64_t{1} << 31) - 1;
constexpr int32_t kMaxHeads = 1 << 14;

Strides dense(int32_t H, int64_t N, int32_t d) {
  return Strides{static_cast<int64_t>(H) * N * d, N * d, d};
}

// Strides of a caller (NULL: dense); false where a stride breaks the
// vectors' alignment.
bool read_strides(const int64_t* st, int32_t H, int64_t N, int32_t d, int64_t step, Strides* out) {
  *out = st ? Strides{st[0], st[1], st[2]} : dense(H, N, d);
  return out->b % step == 0 && out->h % step == 0 && out->n % step == 0;
}

bool check_rope(const ra_rope* r, int32_t d, ra_status* st) {
  *st = RA_ERR_INVALID_ARG;
  if (r->rot < 0 || r->axes < 1 || (r->interleaved != 0 && r->interleaved != 1)) return false;
  *st = RA_ERR_UNSUPPORTED;
  if (r->rot % 8 != 0 || r->rot > RA_MAX_HEAD_DIM || r->rot > d || r->axes > 8) return false;
  *st = RA_ERR_INVALID_ARG;
  for (int i = 0; i < r->rot / 2; ++i)
    if (r->axis[i] >= r->axes) return false;
  *st = RA_OK;
  return true;
}

// Checks shared by the norm's forward and backward; fills the arguments.
ra_status check_norm(const void* q, const int64_t* qs, const void* k, const int64_t* ks,
                     const void* wq, const void* wk, const ra_rope* rope,
                     const int64_t* positions, int32_t B, int32_t Hq, int32_t Hk, int64_t N,
                     int32_t d, float eps, ra_dtype dt, NormArgs* a) {
  if (B < 0 || Hq < 0 || Hk < 0 || N < 0 || d < 1 || std::isnan(eps)) return RA_ERR_INVALID_ARG;
  if (dt != RA_F32 && dt != RA_BF16) return RA_ERR_INVALID_ARG;
  if (eps < 0 && (wq || wk)) return RA_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > RA_MAX_HEAD_DIM || Hq > kMaxHeads || Hk > kMaxHeads)
    return RA_ERR_UNSUPPORTED;
  if (N > kMaxTokens || B * N > kMaxTokens) return RA_ERR_UNSUPPORTED;
  ra_status st;
  if (rope && !check_rope(rope, d, &st)) return st;
  *a = NormArgs{};
  a->N = N;
  a->tokens = B * N;
  a->d = d;
  a->eps = eps;
  const bool empty = a->tokens == 0 || Hq + Hk == 0;
  if (!empty) {
    if ((Hq && !q) || (Hk && !k)) return RA_ERR_INVALID_ARG;
    if (rope && rope->rot && !positions) return RA_ERR_INVALID_ARG;
  }
  const uintptr_t al = dt == RA_BF16 ? 8 : 16;
  if (!aligned(q, al) || !aligned(k, al) || !aligned(wq, al) || !aligned(wk, al) ||
      !aligned(positions, 8))
    return RA_ERR_MISALIGNED;
  if (!read_strides(qs, Hq, N, d, 4, &a->side[0].xs) ||
      !read_strides(ks, Hk, N, d, 4, &a->side[1].xs))
    return RA_ERR_MISALIGNED;
  a->side[0].x = q;
  a->side[1].x = k;
  a->side[0].weight = wq;
  a->side[1].weight = wk;
  a->side[0].heads = Hq;
  a->side[1].heads = Hk;
  a->positions = positions;
  a->has_rope = rope && rope->rot > 0;
  if (a->has_rope) a->rope = *rope;
  return RA_OK;
}

// The cache itself and the sequences of a call; `T` new tokens at most.
ra_status check_cache(const ra_cache* cache, const int32_t* table, int32_t width,
                      const int32_t* lens, int32_t B, int64_t T, ra_dtype dt, PagedArgs* p) {
  if (!cache || B < 0 || T < 0 || width < 0) return RA_ERR_INVALID_ARG;
  if (dt != RA_F32 && dt != RA_BF16) return RA_ERR_INVALID_ARG;
  if (cache->dtype != RA_F32 && cache->dtype != RA_BF16 && cache->dtype != RA_E4M3)
    return RA_ERR_INVALID_ARG;
  if (cache->pages < 0 || cache->heads < 1 || cache->page < 1 || cache->d < 1)
    return RA_ERR_INVALID_ARG;
  if (cache->dtype != RA_E4M3 && cache->dtype != dt) return RA_ERR_UNSUPPORTED;
  if (cache->d % 8 != 0 || cache->d > RA_MAX_HEAD_DIM || cache->heads > kMaxHeads)
    return RA_ERR_UNSUPPORTED;
  if (cache->page < 8 || cache->page > 1024 || (cache->page & (cache->page - 1)) != 0)
    return RA_ERR_UNSUPPORTED;
  // page numbers and TMA coordinates are int32
  if (cache->pages > INT32_MAX || cache->pages * cache->heads > INT32_MAX || B * T > kMaxTokens)
    return RA_ERR_UNSUPPORTED;
  if (cache->pages > 0 && (!cache->k || !cache->v)) return RA_ERR_INVALID_ARG;
  if (cache->dtype == RA_E4M3 && cache->pages > 0 && (!cache->k_exp || !cache->v_exp))
    return RA_ERR_INVALID_ARG;
  if (B > 0 && (!lens || (width > 0 && !table))) return RA_ERR_INVALID_ARG;
  if (!aligned(cache->k, 16) || !aligned(cache->v, 16) || !aligned(cache->k_exp, 8) ||
      !aligned(cache->v_exp, 8) || !aligned(table, 4) || !aligned(lens, 4))
    return RA_ERR_MISALIGNED;
  *p = PagedArgs{};
  p->k = cache->k;
  p->v = cache->v;
  p->ke = cache->k_exp;
  p->ve = cache->v_exp;
  p->pages = cache->pages;
  p->heads = cache->heads;
  p->d = cache->d;
  while ((1 << p->page_shift) < cache->page) ++p->page_shift;
  p->width = width;
  p->table = table;
  p->lens = lens;
  p->B = B;
  p->T = static_cast<int32_t>(T);
  return RA_OK;
}

// Arguments of the attention calls; `a` keeps q = NULL where nothing is to be done.
ra_status check_attention(const void* q, const ra_cache* cache, const int32_t* table, int32_t width,
                          const int32_t* lens, const int32_t* count, const uint8_t* mask, int64_t mask_stride,
                          void* out, float* lse, void* workspace, int64_t workspace_bytes,
                          int64_t (*wanted)(int32_t, int32_t, int32_t, int32_t, int32_t), int32_t B, int32_t Hq,
                          int32_t T, ra_dtype dtype, CacheAttnArgs* a) {
  ra_status st = check_cache(cache, table, width, lens, B, T, dtype, &a->c);
  if (st != RA_OK) return st;
  if (Hq < 0 || Hq % cache->heads != 0) return RA_ERR_INVALID_ARG;
  if (mask && mask_stride != 0 && mask_stride < static_cast<int64_t>(T) * T)
    return RA_ERR_INVALID_ARG;
  if (dtype == RA_BF16 && cache->d != 64 && cache->d != 128) return RA_ERR_UNSUPPORTED;
  if (Hq > kMaxHeads || static_cast<int64_t>(B) * Hq * T > kMaxTokens) return RA_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(count, 4) ||
      !aligned(workspace, 256))
    return RA_ERR_MISALIGNED;
  if (B == 0 || Hq == 0 || T == 0) return RA_OK;
  if (!q || !out || !lse || !workspace) return RA_ERR_INVALID_ARG;
  if (workspace_bytes < wanted(B, Hq, cache->heads, T, cache->d)) return RA_ERR_INVALID_ARG;
  if ((st = device_ready(&a->c.status)) != RA_OK) return st;
  a->c.count = count;
  a->q = q;
  a->mask = mask;
  a->mask_stride = mask_stride;
  a->out = out;
  a->lse = lse;
  a->ws = static_cast<float*>(workspace);
  a->Hq = Hq;
  a->scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(cache->d)));
  a->wait_limit = wait_limit();
  a->stall_cta = stall_cta();
  return RA_OK;
}

// A type that fits the cache, where a call has no tensors beside it.
ra_dtype own_dtype(const ra_cache* cache) { return cache && cache->dtype != RA_E4M3 ? cache->dtype : RA_F32; }

struct Ints {
  const int32_t* p;
  int64_t n;
};
bool overlap(const Ints& x, const Ints& y) {
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.p), y0 = reinterpret_cast<uintptr_t>(y.p);
  return x.n > 0 && y.n > 0 && x0 < y0 + 4 * y.n && y0 < x0 + 4 * x.n;
}

// A table of pages and their counts.
ra_status check_pages(int32_t* ref, int64_t pages, const int32_t* table, const int32_t* held, const int32_t* lens,
                      int32_t width, int32_t page, int32_t B, bool lens_needed, PageTableArgs* a) {
  if (pages < 0 || width < 0 || page < 1 || B < 0) return RA_ERR_INVALID_ARG;
  if (page < 8 || page > 1024 || (page & (page - 1)) != 0) return RA_ERR_UNSUPPORTED;
  if (pages > INT32_MAX || static_cast<int64_t>(B) * width > INT32_MAX) return RA_ERR_UNSUPPORTED;
  if (B > 0 && (!held || (lens_needed && !lens) || (width > 0 && !table) || (pages > 0 && !ref)))
    return RA_ERR_INVALID_ARG;
  if (!aligned(ref, 4) || !aligned(table, 4) || !aligned(held, 4) || !aligned(lens, 4)) return RA_ERR_MISALIGNED;
  *a = PageTableArgs{};
  a->ref = ref;
  a->pages = pages;
  a->table = const_cast<int32_t*>(table);
  a->held = const_cast<int32_t*>(held);
  a->lens = lens;
  a->width = width;
  a->B = B;
  while ((1 << a->page_shift) < page) ++a->page_shift;
  return RA_OK;
}

}  // namespace
}  // namespace ra

using namespace ra;

extern "C" {

RA_API ra_status ra_rope_init(ra_rope* rope, const double* inv_freq, const int32_t* axis,
                              int32_t rot, int32_t axes, int32_t interleaved) {
  if (!rope || rot < 0 || axes < 1 || (interleaved != 0 && interleaved != 1))
    return RA_ERR_INVALID_ARG;
  if (rot > 0 && !inv_freq) return RA_ERR_INVALID_ARG;
  if (rot % 8 != 0 || rot > RA_MAX_HEAD_DIM || axes > 8) return RA_ERR_UNSUPPORTED;
  ra_rope r{};
  r.rot = rot;
  r.axes = axes;
  r.interleaved = interleaved;
  // 1 / (2 pi) = kInv * 2^-130, kInv = kInvHi * 2^64 + kInvLo.
  constexpr uint64_t kInvHi = 0xA2F9836E4E441529ull, kInvLo = 0xFC2757D1F534DDC1ull;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = inv_freq[i];
    if (!(std::fabs(f) < 2147483648.0)) return RA_ERR_INVALID_ARG;
    if (axis && (axis[i] < 0 || axis[i] >= axes)) return RA_ERR_INVALID_ARG;
    r.axis[i] = static_cast<uint8_t>(axis ? axis[i] : 0);
    int ex = 0;
    const double fr = std::frexp(std::fabs(f), &ex);  // f = m * 2^(ex - 53)
    const uint64_t m = static_cast<uint64_t>(std::ldexp(fr, 53));
    // m * kInv in three 64-bit words, then * 2^(ex - 53 - 130 + 64), rounded
    using u128 = unsigned __int128;
    const u128 lo = static_cast<u128>(m) * kInvLo, hi = static_cast<u128>(m) * kInvHi;
    const u128 mid = hi + static_cast<uint64_t>(lo >> 64);
    const uint64_t w[4] = {static_cast<uint64_t>(lo), static_cast<uint64_t>(mid),
                           static_cast<uint64_t>(mid >> 64), 0};
    const int shift = 119 - ex;  // > 87, since ex <= 31
    uint64_t turns = 0;
    if (shift <= 192) {
      auto bits = [&](int at) {  // 64 bits of the product from bit `at` on
        const int j = at / 64, z = at % 64;
        const uint64_t a0 = j < 4 ? w[j] : 0, a1 = j + 1 < 4 ? w[j + 1] : 0;
        return z ? (a0 >> z) | (a1 << (64 - z)) : a0;
      };
      turns = bits(shift) + (bits(shift - 1) & 1);
    }
    r.turns[i] = f < 0 ? 0 - turns : turns;
  }
  *rope = r;
  return RA_OK;
}

RA_API ra_status ra_qk_norm_rope(const void* q, const int64_t* q_strides, const void* k,
                                 const int64_t* k_strides, const void* q_weight,
                                 const void* k_weight, const ra_rope* rope,
                                 const int64_t* positions, void* q_out, void* k_out, int32_t B,
                                 int32_t Hq, int32_t Hk, int64_t N, int32_t d, float eps,
                                 ra_dtype dtype, ra_stream_t stream) {
  RA_TRACE("ra_qk_norm_rope");
  NormArgs a;
  ra_status st = check_norm(q, q_strides, k, k_strides, q_weight, k_weight, rope, positions, B, Hq,
                            Hk, N, d, eps, dtype, &a);
  if (st != RA_OK) return st;
  if (a.tokens == 0 || Hq + Hk == 0) return RA_OK;
  if ((Hq && !q_out) || (Hk && !k_out)) return RA_ERR_INVALID_ARG;
  const uintptr_t al = dtype == RA_BF16 ? 8 : 16;
  if (!aligned(q_out, al) || !aligned(k_out, al)) return RA_ERR_MISALIGNED;
  a.side[0].y = q_out;
  a.side[1].y = k_out;
  a.side[0].ys = dense(Hq, N, d);
  a.side[1].ys = dense(Hk, N, d);
  int* status = nullptr;
  if ((st = device_ready(&status)) != RA_OK) return st;
  return launched(launch_norm_rope(a, dtype == RA_BF16, cu(stream)));
}

RA_API int64_t ra_qk_norm_rope_backward_workspace_bytes(int32_t d) {
  if (d < 1 || d % 8 != 0 || d > RA_MAX_HEAD_DIM) return -1;
  return static_cast<int64_t>(kNormBackwardBlocks) * 2 * d * 4;
}

RA_API ra_status ra_qk_norm_rope_backward(
    const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
    const void* q_weight, const void* k_weight, const ra_rope* rope, const int64_t* positions,
    const void* dq_out, const void* dk_out, void* dq, const int64_t* dq_strides, void* dk,
    const int64_t* dk_strides, float* dq_weight, float* dk_weight, void* workspace,
    int64_t workspace_bytes, int32_t B, int32_t Hq, int32_t Hk, int64_t N, int32_t d, float eps,
    ra_dtype dtype, ra_stream_t stream) {
  RA_TRACE("ra_qk_norm_rope_backward");
  NormArgs a;
  ra_status st = check_norm(q, q_strides, k, k_strides, q_weight, k_weight, rope, positions, B, Hq,
                            Hk, N, d, eps, dtype, &a);
  if (st != RA_OK) return st;
  const bool weights = q_weight || k_weight;
  if (!q_weight != !dq_weight || !k_weight != !dk_weight) return RA_ERR_INVALID_ARG;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(workspace, 16))
    return RA_ERR_MISALIGNED;
  const bool empty = a.tokens == 0 || Hq + Hk == 0;
  if (!empty) {
    if ((Hq && (!dq_out || !dq)) || (Hk && (!dk_out || !dk))) return RA_ERR_INVALID_ARG;
    if (weights &&
        (!workspace || workspace_bytes < ra_qk_norm_rope_backward_workspace_bytes(d)))
      return RA_ERR_INVALID_ARG;
  }
  const uintptr_t al = dtype == RA_BF16 ? 8 : 16;
  if (!aligned(dq_out, al) || !aligned(dk_out, al) || !aligned(dq, al) || !aligned(dk, al))
    return RA_ERR_MISALIGNED;
  if (!read_strides(dq_strides, Hq, N, d, 4, &a.side[0].ys) ||
      !read_strides(dk_strides, Hk, N, d, 4, &a.side[1].ys))
    return RA_ERR_MISALIGNED;
  for (const NormSide& s : a.side)  // a gradient row per input row
    if (!empty && s.heads > 0 &&
        ((B > 1 && s.ys.b == 0) || (s.heads > 1 && s.ys.h == 0) || (N > 1 && s.ys.n == 0)))
      return RA_ERR_INVALID_ARG;
  if (empty && !weights) return RA_OK;
  int* status = nullptr;
  if ((st = device_ready(&status)) != RA_OK) return st;
  if (empty) {  // no row: the weights' gradients are zero
    if (dq_weight && (st = launched(cudaMemsetAsync(dq_weight, 0, d * 4, cu(stream)))) != RA_OK)
      return st;
    return dk_weight ? launched(cudaMemsetAsync(dk_weight, 0, d * 4, cu(stream))) : RA_OK;
  }
  a.side[0].dy = dq_out;
  a.side[1].dy = dk_out;
  a.side[0].y = dq;
  a.side[1].y = dk;
  a.side[0].dweight = dq_weight;
  a.side[1].dweight = dk_weight;
  a.partial = weights ? static_cast<float*>(workspace) : nullptr;
  return launched(launch_norm_rope_backward(a, dtype == RA_BF16, cu(stream)));
}

RA_API ra_status ra_cache_write(const ra_cache* cache, const void* k, const int64_t* k_strides,
                                const void* v, const int64_t* v_strides, const int32_t* table,
                                int32_t width, const int32_t* lens, const int32_t* count,
                                int32_t B, int32_t T, ra_dtype dtype, ra_stream_t stream) {
  RA_TRACE("ra_cache_write");
  CacheCopyArgs a{};
  ra_status st = check_cache(cache, table, width, lens, B, T, dtype, &a.c);
  if (st != RA_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(count, 4)) return RA_ERR_MISALIGNED;
  const int64_t step = dtype == RA_BF16 ? 8 : 4;
  if (!read_strides(k_strides, cache->heads, T, cache->d, step, &a.ks) ||
      !read_strides(v_strides, cache->heads, T, cache->d, step, &a.vs))
    return RA_ERR_MISALIGNED;
  if (B == 0 || T == 0) return RA_OK;
  if (!k || !v) return RA_ERR_INVALID_ARG;
  if ((st = device_ready(&a.c.status)) != RA_OK) return st;
  a.c.count = count;
  a.k = const_cast<void*>(k);
  a.v = const_cast<void*>(v);
  a.n = T;
  return launched(launch_cache_write(a, dtype, cache->dtype, cu(stream)));
}

RA_API ra_status ra_cache_read(const ra_cache* cache, const int32_t* table, int32_t width,
                               const int32_t* lens, int64_t first, int64_t n, void* k, void* v,
                               int32_t B, ra_dtype dtype, ra_stream_t stream) {
  RA_TRACE("ra_cache_read");
  CacheCopyArgs a{};
  if (first < 0 || n < 0) return RA_ERR_INVALID_ARG;
  ra_status st = check_cache(cache, table, width, lens, B, 0, dtype, &a.c);
  if (st != RA_OK) return st;
  if (n > kMaxTokens || B * n > kMaxTokens) return RA_ERR_UNSUPPORTED;
  if (!aligned(k, 16) || !aligned(v, 16)) return RA_ERR_MISALIGNED;
  if (B == 0 || n == 0) return RA_OK;
  if (!k || !v) return RA_ERR_INVALID_ARG;
  if ((st = device_ready(&a.c.status)) != RA_OK) return st;
  a.k = k;
  a.v = v;
  // lens is an int32: behind 2^31 every row is 0, and first + n must not wrap
  a.first = first < kMaxTokens + 1 ? first : kMaxTokens + 1;
  a.n = n;
  return launched(launch_cache_read(a, dtype, cache->dtype, cu(stream)));
}

RA_API int64_t ra_cache_attention_workspace_bytes(int32_t B, int32_t Hq, int32_t heads, int32_t T,
                                                  int32_t d) {
  if (B < 0 || Hq < 0 || heads < 1 || T < 0 || d < 1 || d > RA_MAX_HEAD_DIM || Hq % heads != 0)
    return -1;
  return cache_attention_workspace_bytes(B, Hq, heads, T, d);
}

RA_API ra_status ra_cache_attention(const void* q, const ra_cache* cache, const int32_t* table,
                                    int32_t width, const int32_t* lens, const int32_t* count,
                                    const uint8_t* mask, int64_t mask_stride, void* out,
                                    float* lse, void* workspace, int64_t workspace_bytes,
                                    int32_t B, int32_t Hq, int32_t T, ra_dtype dtype,
                                    ra_stream_t stream) {
  RA_TRACE("ra_cache_attention");
  CacheAttnArgs a{};
  const ra_status st = check_attention(q, cache, table, width, lens, count, mask, mask_stride, out, lse, workspace,
                                       workspace_bytes, cache_attention_workspace_bytes, B, Hq, T, dtype, &a);
  return st != RA_OK || !a.q ? st : launched(launch_cache_attention(a, dtype, cache->dtype, cu(stream)));
}

RA_API int64_t ra_cache_attention_shared_workspace_bytes(int32_t B, int32_t Hq, int32_t heads, int32_t T,
                                                         int32_t d) {
  if (B < 0 || Hq < 0 || heads < 1 || T < 0 || d < 1 || d > RA_MAX_HEAD_DIM || Hq % heads != 0)
    return -1;
  return cache_attention_shared_workspace_bytes(B, Hq, heads, T, d);
}

RA_API ra_status ra_cache_attention_shared(const void* q, const ra_cache* cache, const int32_t* table,
                                           int32_t width, const int32_t* lens, const int32_t* shared,
                                           const int32_t* count, const uint8_t* mask, int64_t mask_stride,
                                           void* out, float* lse, void* workspace, int64_t workspace_bytes,
                                           int32_t B, int32_t Hq, int32_t T, ra_dtype dtype, ra_stream_t stream) {
  RA_TRACE("ra_cache_attention_shared");
  CacheAttnArgs a{};
  if (!shared && B > 0 && Hq > 0 && T > 0) return RA_ERR_INVALID_ARG;
  if (!aligned(shared, 4)) return RA_ERR_MISALIGNED;
  const ra_status st = check_attention(q, cache, table, width, lens, count, mask, mask_stride, out, lse, workspace,
                                       workspace_bytes, cache_attention_shared_workspace_bytes, B, Hq, T, dtype, &a);
  if (st != RA_OK || !a.q) return st;
  return launched(launch_cache_attention_shared(a, shared, dtype, cache->dtype, cu(stream)));
}

RA_API ra_status ra_pages_fork(int32_t* ref, int64_t pages, const int32_t* table, const int32_t* held,
                               const int32_t* lens, int32_t width, int32_t page, int32_t B, const int32_t* source,
                               int32_t n, int32_t* table_out, int32_t* held_out, int32_t* lens_out,
                               ra_stream_t stream) {
  RA_TRACE("ra_pages_fork");
  PageTableArgs a;
  ra_status st = check_pages(ref, pages, table, held, lens, width, page, B, true, &a);
  if (st != RA_OK) return st;
  if (n < 0) return RA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n) * width > INT32_MAX) return RA_ERR_UNSUPPORTED;
  if (!aligned(source, 4) || !aligned(table_out, 4) || !aligned(held_out, 4) || !aligned(lens_out, 4))
    return RA_ERR_MISALIGNED;
  if (n == 0) return RA_OK;
  if (!source || (width > 0 && !table_out) || !held_out || !lens_out) return RA_ERR_INVALID_ARG;
  // what is written would be read by another row's block
  const Ints out[] = {{table_out, static_cast<int64_t>(n) * width}, {held_out, n}, {lens_out, n}};
  const Ints in[] = {{ref, pages}, {table, static_cast<int64_t>(B) * width}, {held, B}, {lens, B}, {source, n}};
  for (const Ints& x : out)
    for (const Ints& y : in)
      if (overlap(x, y)) return RA_ERR_INVALID_ARG;
  if ((st = device_ready(&a.status)) != RA_OK) return st;
  return launched(launch_pages_fork(a, source, n, table_out, held_out, lens_out, cu(stream)));
}

RA_API ra_status ra_pages_reserve(int32_t* ref, int64_t pages, int32_t* table, int32_t* held, const int32_t* lens,
                                  const int32_t* count, int32_t width, int32_t page, int32_t B, int32_t T,
                                  int32_t* granted, int32_t* src, int32_t* dst, ra_stream_t stream) {
  RA_TRACE("ra_pages_reserve");
  PageTableArgs a;
  ra_status st = check_pages(ref, pages, table, held, lens, width, page, B, true, &a);
  if (st != RA_OK) return st;
  if (T < 0) return RA_ERR_INVALID_ARG;
  if (B > kReserveSequences) return RA_ERR_UNSUPPORTED;
  if (!aligned(count, 4) || !aligned(granted, 4) || !aligned(src, 4) || !aligned(dst, 4)) return RA_ERR_MISALIGNED;
  if (B == 0) return RA_OK;
  if (!granted || !src || !dst) return RA_ERR_INVALID_ARG;
  if ((st = device_ready(&a.status)) != RA_OK) return st;
  return launched(launch_pages_reserve(a, count, T, granted, src, dst, cu(stream)));
}

RA_API ra_status ra_pages_trim(int32_t* ref, int64_t pages, int32_t* table, int32_t* held, const int32_t* lens,
                               int32_t width, int32_t page, int32_t B, ra_stream_t stream) {
  RA_TRACE("ra_pages_trim");
  PageTableArgs a;
  ra_status st = check_pages(ref, pages, table, held, lens, width, page, B, false, &a);
  if (st != RA_OK) return st;
  if (B == 0) return RA_OK;
  if ((st = device_ready(&a.status)) != RA_OK) return st;
  return launched(launch_pages_trim(a, cu(stream)));
}

RA_API ra_status ra_cache_copy(const ra_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                               ra_stream_t stream) {
  RA_TRACE("ra_cache_copy");
  PagedArgs c;
  if (n < 0) return RA_ERR_INVALID_ARG;
  ra_status st = check_cache(cache, nullptr, 0, nullptr, 0, 0, own_dtype(cache), &c);
  if (st != RA_OK) return st;
  if (!aligned(src, 4) || !aligned(dst, 4)) return RA_ERR_MISALIGNED;
  if (n == 0) return RA_OK;
  if (!src || !dst) return RA_ERR_INVALID_ARG;
  if ((st = device_ready(&c.status)) != RA_OK) return st;
  return launched(launch_cache_copy(c, cache->dtype, src, dst, n, cu(stream)));
}

RA_API ra_status ra_cache_compact(const ra_cache* cache, const int32_t* table, int32_t width, const int32_t* lens,
                                  const int32_t* path, const int32_t* kept, int32_t B, int32_t T,
                                  ra_stream_t stream) {
  RA_TRACE("ra_cache_compact");
  PagedArgs c;
  ra_status st = check_cache(cache, table, width, lens, B, T, own_dtype(cache), &c);
  if (st != RA_OK) return st;
  if (!aligned(path, 4) || !aligned(kept, 4)) return RA_ERR_MISALIGNED;
  if (B == 0 || T == 0) return RA_OK;
  if (!path || !kept) return RA_ERR_INVALID_ARG;
  if ((st = device_ready(&c.status)) != RA_OK) return st;
  c.count = kept;
  return launched(launch_cache_compact(c, cache->dtype, path, cu(stream)));
}

RA_API ra_status ra_verify_drafts(const void* probs, const void* draft_probs, const int64_t* tokens,
                                  const int32_t* parent, const int32_t* count, const float* uniform, int32_t* path,
                                  int32_t* kept, int64_t* token, int32_t B, int32_t T, int64_t V, ra_dtype dtype,
                                  ra_stream_t stream) {
  RA_TRACE("ra_verify_drafts");
  if (B < 0 || T < 1 || V < 1) return RA_ERR_INVALID_ARG;
  if (dtype != RA_F32 && dtype != RA_BF16) return RA_ERR_INVALID_ARG;
  if (T > kVerifyNodes || V > INT32_MAX || B > (1 << 24)) return RA_ERR_UNSUPPORTED;
  if (!aligned(probs, 16) || !aligned(draft_probs, 16) || !aligned(tokens, 8) || !aligned(token, 8) ||
      !aligned(parent, 4) || !aligned(count, 4) || !aligned(uniform, 4) || !aligned(path, 4) || !aligned(kept, 4))
    return RA_ERR_MISALIGNED;
  if (B == 0) return RA_OK;
  if (!probs || !tokens || !uniform || !path || !kept || !token) return RA_ERR_INVALID_ARG;
  int* status = nullptr;
  const ra_status st = device_ready(&status);
  if (st != RA_OK) return st;
  const VerifyArgs a{probs, draft_probs, tokens, parent, count, uniform, path, kept, token, B, T, V};
  return launched(launch_verify(a, dtype == RA_BF16, cu(stream)));
}

}  // extern "C"
