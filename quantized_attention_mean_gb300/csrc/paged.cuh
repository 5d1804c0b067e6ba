// View of a paged key-value cache and what the kernels over it share.
//
// A page holds page_size token slots of every key/value head; row b of the page table lists the
// pages of sequence b, whose token slot t lies in page table[b][t / page_size] at t % page_size.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/sageattn.h"
#include "problem.cuh"

namespace sage {

constexpr int kDevPage = 13;  // SAGE_ERR_PAGE
constexpr int64_t kMostSlots = 0x7fff0000;  // of a sequence: the kernels look some thousand slots past the last in 32 bits

struct PagedView {
  void* k; int64_t k_sp, k_sh, k_st;  // element strides of (page, head, token slot)
  void* v; int64_t v_sp, v_sh, v_st;
  const int* table; int64_t table_stride;
  const int* lens;
  float* mass;  // [num_pages, hkv, page_size] or null
  int* pos;     // likewise
  int batch, hkv, d, page_size, num_pages, max_pages;
};

// Host: checks a cache description and its layout; *vec: every K and V row of whole 16-byte loads.
int make_paged_view(const sage_paged_cache* cache, int batch, int heads_kv, int head_dim, int dtype,
                    int tensor_layout, PagedView* view, bool* vec);

// Index of (page, head, slot) in the mass and position planes.
__device__ __forceinline__ int64_t plane_at(const PagedView& c, int page, int h, int slot) {
  return ((int64_t)page * c.hkv + h) * c.page_size + slot;
}

// Length of sequence b, or -1 where it lies outside of the table's room or of max_len.
__device__ __forceinline__ int checked_len(const PagedView& c, int b, int64_t max_len) {
  const int64_t n = __ldg(&c.lens[b]);
  return n >= 0 && n <= (int64_t)c.max_pages * c.page_size && n <= max_len ? (int)n : -1;
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16-byte asynchronous copy to shared memory; bytes beyond `src_bytes` are written as zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace sage
