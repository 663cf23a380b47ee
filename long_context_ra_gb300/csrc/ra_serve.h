// Internal interface of the calls around the attention: the norm and
// rotation of queries and keys, and the paged K/V cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ra.h"

namespace ra {

// Element strides of a [B, H, N, d] tensor whose d is contiguous.
struct Strides {
  int64_t b, h, n;
};

struct NormSide {
  const void* x;       // input rows
  const void* dy;      // backward: gradient of the output rows (dense)
  void* y;             // forward: output rows; backward: gradient of x
  const void* weight;  // [d] or NULL
  float* dweight;      // backward: fp32 [d]
  Strides xs, ys;
  int32_t heads;
};

struct NormArgs {
  NormSide side[2];  // q, k
  const int64_t* positions;
  int64_t N, tokens;  // tokens = B * N
  int32_t d;
  float eps;      // < 0: no norm
  float* partial;  // backward: [blocks, 2, d] sums of dw
  int32_t has_rope;
  ra_rope rope;
};

// Blocks of the backward, and so the rows of its partial sums.
constexpr int kNormBackwardBlocks = 304;  // two per SM

cudaError_t launch_norm_rope(const NormArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_norm_rope_backward(const NormArgs& a, bool bf16, cudaStream_t s);

// A cache as the kernels see it, with the sequences of one call.
struct PagedArgs {
  void* k;
  void* v;
  uint8_t* ke;  // exponent bytes (8-bit cache)
  uint8_t* ve;
  int64_t pages;
  int32_t heads, d;
  int32_t page_shift;  // log2 of the rows of a page
  int32_t width;       // pages per row of the table
  const int32_t* table;
  const int32_t* lens;
  const int32_t* count;  // NULL: T each
  int32_t B, T;
  int* status;
};

// TMA view of one side of a cache, [pages x heads, page, d], with boxes of
// box_rows rows: 64 bf16 columns with the 128-byte swizzle of the MMA
// operands, or whole rows of bytes.
bool encode_pages(CUtensorMap* map, const void* ptr, const PagedArgs& c, int box_rows, bool bytes);
// TMA view of dense bf16 rows [rows, d] with boxes of 128 rows of 64 columns, swizzled alike.
bool encode_rows(CUtensorMap* map, const void* ptr, int64_t rows, int d);
// The same with boxes of one row, for loads that gather rows.
bool encode_single_rows(CUtensorMap* map, const void* ptr, int64_t rows, int d);

struct CacheCopyArgs {
  PagedArgs c;
  void* k;  // the dense side: [B, heads, n, d]
  void* v;
  Strides ks, vs;
  int64_t first, n;
};

// Element types of the dense side (f32 or bf16) and of the cache.
cudaError_t launch_cache_write(const CacheCopyArgs& a, ra_dtype dense, ra_dtype held,
                               cudaStream_t s);
cudaError_t launch_cache_read(const CacheCopyArgs& a, ra_dtype dense, ra_dtype held,
                              cudaStream_t s);

// Rows of page numbers, and how many rows hold each page.
struct PageTableArgs {
  int32_t* ref;  // [pages]
  int64_t pages;
  int32_t* table;  // [B, width]
  int32_t* held;   // [B] columns that hold a page
  const int32_t* lens;
  int32_t width, B;
  int32_t page_shift;
  int* status;
};

// Sequences of one reservation: five bytes of shared memory each.
constexpr int kReserveSequences = 8192;

cudaError_t launch_pages_fork(const PageTableArgs& a, const int32_t* source, int32_t n, int32_t* table_out,
                              int32_t* held_out, int32_t* lens_out, cudaStream_t s);
cudaError_t launch_pages_reserve(const PageTableArgs& a, const int32_t* count, int32_t T, int32_t* granted,
                                 int32_t* src, int32_t* dst, cudaStream_t s);
cudaError_t launch_pages_trim(const PageTableArgs& a, cudaStream_t s);
cudaError_t launch_cache_copy(const PagedArgs& c, ra_dtype held, const int32_t* src, const int32_t* dst, int32_t n,
                              cudaStream_t s);
// The kept tokens of a sequence are c.count.
cudaError_t launch_cache_compact(const PagedArgs& c, ra_dtype held, const int32_t* path, cudaStream_t s);

// Drafts of one call: their tokens, parents and probabilities lie in shared memory.
constexpr int kVerifyNodes = 1024;

struct VerifyArgs {
  const void* probs;  // [B, T, V]
  const void* draft;  // the same, or NULL
  const int64_t* tokens;
  const int32_t* parent;  // NULL: t - 1
  const int32_t* count;   // NULL: T
  const float* uniform;
  int32_t* path;
  int32_t* kept;
  int64_t* token;
  int32_t B, T;
  int64_t V;
};

cudaError_t launch_verify(const VerifyArgs& a, bool bf16, cudaStream_t s);

struct CacheAttnArgs {
  PagedArgs c;
  const void* q;  // [B, Hq, T, d]
  const uint8_t* mask;
  int64_t mask_stride;
  void* out;
  float* lse;
  float* ws;  // partial states
  int32_t Hq;
  float scale_log2;  // log2(e) / sqrt(d)
  int64_t wait_limit;
  int64_t stall_cta;
};

cudaError_t launch_cache_attention(const CacheAttnArgs& a, ra_dtype dense, ra_dtype held,
                                   cudaStream_t s);
// `shared` [B]: tokens that a sequence has in common with the one before it.
cudaError_t launch_cache_attention_shared(const CacheAttnArgs& a, const int32_t* shared, ra_dtype dense,
                                          ra_dtype held, cudaStream_t s);
int64_t cache_attention_shared_workspace_bytes(int32_t B, int32_t Hq, int32_t heads, int32_t T,
                                               int32_t d);
int64_t cache_attention_workspace_bytes(int32_t B, int32_t Hq, int32_t heads, int32_t T,
                                        int32_t d);

}  // namespace ra
