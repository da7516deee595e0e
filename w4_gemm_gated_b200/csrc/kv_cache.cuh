// The paged key-value cache as the kernels see it (spear_kv_cache, validated).
#pragma once

#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace spear {

struct KvView {
  int kind, n_pages, log_page, page_size, heads, dim;
  uint8_t* k;
  uint8_t* v;
  __half* ks;
  __half* vs;
  long long page_stride, scale_stride;  // bytes, elements
  uint32_t page_step, scale_step;       // the same in 16 bytes
};

// Bits of a stored value.
__host__ __device__ constexpr int kv_bits(int kind) {
  return kind == SPEAR_KV_BF16 ? 16 : kind == SPEAR_KV_INT8 ? 8 : 4;
}

// Validate a public cache description; SPEAR_OK or the status to return.
int check_kv_cache(const spear_kv_cache* c, KvView* out);

inline bool ptr_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Whether np bytes from p and nq bytes from q share one (NULL: no).
inline bool buffers_meet(const void* p, uintptr_t np, const void* q, uintptr_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + nq && b < a + np;
}

// Distance to a page, in 16-byte steps.
__device__ __forceinline__ long long page_at(uint32_t page, uint32_t step) { return (long long)((uint64_t)page * step); }

// Start of a kernel launched by launch_after: its blocks come to the SMs while
// the previous kernel in the stream ends (1 us saved between two of them), and
// wait here until all that it wrote is visible.  What such a kernel reads may
// have been written while it was on its way, so it is read by plain loads, not
// through the read-only path (__ldg, const __restrict__).
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// f(kind, dim) as a compile-time pair.
template <class F>
void for_kind_dim(int kind, int dim, F f) {
  auto with_dim = [&](auto kc) {
    if (dim == 64) f(kc, std::integral_constant<int, 64>{});
    if (dim == 128) f(kc, std::integral_constant<int, 128>{});
    if (dim == 256) f(kc, std::integral_constant<int, 256>{});
  };
  if (kind == SPEAR_KV_BF16) with_dim(std::integral_constant<int, SPEAR_KV_BF16>{});
  if (kind == SPEAR_KV_INT8) with_dim(std::integral_constant<int, SPEAR_KV_INT8>{});
  if (kind == SPEAR_KV_INT4) with_dim(std::integral_constant<int, SPEAR_KV_INT4>{});
}

}  // namespace spear
