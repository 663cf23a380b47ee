// Shared by the attention kernels over the paged cache: the query rows of a
// unit, the visibility of keys, and the plan that divides the work.
#pragma once

#include "ra_paged.cuh"

namespace ra {

constexpr float kLn2F = 0.6931471805599453f;

// One launch's plan: how many query rows a unit holds and how its key tiles
// are divided.  Partial states are [slots][rows][2] (m in log2 units, l)
// followed by [slots][rows][d] (o); the many-row kernel, whose threads hold a
// row each, writes o as [slots][d / 4][rows][4].
struct AttnPlan {
  Division div;
  int rows;       // query rows per unit
  int row_tiles;  // units per (sequence, key head)
};

// Query rows of one key head: g heads x T tokens, token fastest, which is
// the order they have in q, out and lse.
__host__ __device__ __forceinline__ int64_t head_rows(const CacheAttnArgs& a) {
  return static_cast<int64_t>(a.Hq / a.c.heads) * a.c.T;
}

__device__ __forceinline__ float* slot_ml(const CacheAttnArgs& a, const AttnPlan& p, int slot) {
  return a.ws + static_cast<int64_t>(slot) * p.rows * 2;
}
__device__ __forceinline__ float* slot_o(const CacheAttnArgs& a, const AttnPlan& p, int slot) {
  return a.ws + static_cast<int64_t>(2 * p.div.ctas) * p.rows * 2 +
         static_cast<int64_t>(slot) * p.rows * a.c.d;
}

// The join is launched while the kernel that writes the parts still runs
// (programmatic dependent launch): the kernel allows it at its start, the join
// works out where its rows lie and then waits for the kernel's end.
__device__ __forceinline__ void allow_join() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_parts() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Whether query t sees the key at position pos of its sequence.
__device__ __forceinline__ bool sees(const CacheAttnArgs& a, const SeqInfo& s, int b, int t,
                                     int64_t pos) {
  if (t >= s.cnt) return false;
  if (pos < s.len) return true;
  const int64_t j = pos - s.len;
  if (j >= s.cnt) return false;
  if (!a.mask) return j <= t;
  return a.mask[b * a.mask_stride + static_cast<int64_t>(t) * a.c.T + j] != 0;
}

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(at));
  return x;
}

// CTAs of the kernels, which fix the size of the workspace.
constexpr int kFfmaCtas = 608;
constexpr int kDecodeCtas = 304;  // two per SM
constexpr int kDecodeRows = 16;
constexpr int kTreeCtas = 152;  // one per SM

cudaError_t launch_cache_decode(const CacheAttnArgs& a, bool k8, cudaStream_t s);
cudaError_t launch_cache_tree(const CacheAttnArgs& a, bool k8, cudaStream_t s);

// Joins the parts of the units that several CTAs shared.
cudaError_t launch_cache_attn_join(const CacheAttnArgs& a, const AttnPlan& p, bool bf16,
                                   cudaStream_t s);
cudaError_t launch_cache_tree_join(const CacheAttnArgs& a, const AttnPlan& p, cudaStream_t s);

}  // namespace ra
