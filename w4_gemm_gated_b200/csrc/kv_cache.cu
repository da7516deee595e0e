// Paged key-value cache: quantising tokens as they are written, and reading
// them back.
//
// A row is one token's head_dim values of one head, keys or values.  Its fp16
// scale is s = fp16(max|w| / Q) and its codes are rint(w / s), Q = 127 or 7
// (include/spear.h has the exact rule); it reads back as bf16(c * s).  Both
// calls are copies with a few operations per value, bound by HBM at large
// sizes and by the launch at a decode step's.
#include "kv_cache.cuh"

namespace spear {

int check_kv_cache(const spear_kv_cache* c, KvView* out) {
  if (!c) return set_error(SPEAR_ERR_INVALID_ARG, "cache is NULL");
  const size_t page_bytes = spear_kv_page_bytes(c->kind, c->page_size, c->n_heads, c->head_dim);
  if (page_bytes == 0)
    return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE,
                     "cache kind=%d page_size=%d n_heads=%d head_dim=%d: kinds 0 to 2, pages of a power of two from 16 "
                     "to 1024 tokens, 1 to 1024 heads of 64, 128 or 256",
                     c->kind, c->page_size, c->n_heads, c->head_dim);
  if (c->n_pages < 1 || (long long)c->n_pages * c->page_size > 0x7fffffffLL)
    return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "n_pages=%d: the cache must hold 1 page and less than 2^31 tokens",
                     c->n_pages);
  const bool quant = c->kind != SPEAR_KV_BF16;
  if (!c->k || !c->v || (quant && (!c->k_scales || !c->v_scales)))
    return set_error(SPEAR_ERR_INVALID_ARG, "cache has a NULL pointer");
  if (!ptr_aligned16(c->k) || !ptr_aligned16(c->v) ||
      (quant && (!ptr_aligned16(c->k_scales) || !ptr_aligned16(c->v_scales))))
    return set_error(SPEAR_ERR_ALIGNMENT, "cache device pointers must be 16-byte aligned");
  const long long page_scales = (long long)c->n_heads * c->page_size;
  if (c->page_stride != 0 && (c->page_stride < (long long)page_bytes || c->page_stride % 16))
    return set_error(SPEAR_ERR_INVALID_ARG, "page_stride=%lld: 0, or a multiple of 16 of at least %zu bytes",
                     c->page_stride, page_bytes);
  if (quant && c->scale_stride != 0 && (c->scale_stride < page_scales || c->scale_stride % 8))
    return set_error(SPEAR_ERR_INVALID_ARG, "scale_stride=%lld: 0, or a multiple of 8 of at least %lld",
                     c->scale_stride, page_scales);
  if (c->page_stride >> 36 || c->scale_stride >> 35)
    return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "pages lie more than 2^36 bytes apart");
  out->kind = c->kind;
  out->n_pages = c->n_pages;
  out->page_size = c->page_size;
  out->log_page = 31 - __builtin_clz((unsigned)c->page_size);
  out->heads = c->n_heads;
  out->dim = c->head_dim;
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->ks = quant ? reinterpret_cast<__half*>(c->k_scales) : nullptr;
  out->vs = quant ? reinterpret_cast<__half*>(c->v_scales) : nullptr;
  out->page_stride = c->page_stride ? c->page_stride : (long long)page_bytes;
  out->scale_stride = c->scale_stride ? c->scale_stride : page_scales;
  out->page_step = (uint32_t)(out->page_stride / 16);
  out->scale_step = (uint32_t)(out->scale_stride / 8);
  return SPEAR_OK;
}

__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }

// One lane per 8 values (16 bytes of bf16), DIM / 8 lanes per row, one row
// per lane group; blockIdx.y: keys or values.
template <int KIND, int DIM>
__global__ void __launch_bounds__(256) kv_write_kernel(KvView c, const __nv_bfloat16* __restrict__ k, long long ld_k,
                                                       const __nv_bfloat16* __restrict__ v, long long ld_v,
                                                       const int* __restrict__ slots, int n, WsHeader* hdr) {
  constexpr int LPR = DIM / 8;
  const bool is_v = blockIdx.y != 0;
  const int lane_r = threadIdx.x % LPR;
  const long long row = (long long)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (row >= (long long)n * c.heads) return;  // whole lane groups leave together
  const int tok = (int)(row / c.heads), head = (int)(row % c.heads);
  const int slot = slots[tok];
  const int page = slot >> c.log_page, off = slot & (c.page_size - 1);
  if (slot < 0) return;
  if (page >= c.n_pages) {
    if (lane_r == 0) report_status(hdr, SPEAR_ERR_DEVICE_CHECK);
    return;
  }
  const __nv_bfloat16* src = is_v ? v + tok * ld_v : k + tok * ld_k;
  const uint4 w = *reinterpret_cast<const uint4*>(src + head * DIM + lane_r * 8);
  const long long prow = (long long)head * c.page_size + off;  // row inside the page
  uint8_t* dst = (is_v ? c.v : c.k) + page * c.page_stride + (prow * DIM + lane_r * 8) * kv_bits(KIND) / 8;
  if constexpr (KIND == SPEAR_KV_BF16) {
    *reinterpret_cast<uint4*>(dst) = w;
    return;
  }
  constexpr float Q = KIND == SPEAR_KV_INT8 ? 127.f : 7.f;
  // max of the magnitudes as 16-bit patterns: a NaN's pattern is above infinity's
  uint32_t m2 = absmax2(absmax2(absmax2(absmax2(0u, w.x), w.y), w.z), w.w);
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  // this row's lanes (other rows of the warp may have left)
  const unsigned group = (LPR == 32 ? 0xFFFFFFFFu : (1u << LPR) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(group, m, d, LPR));
  __half hs = __float2half_rn(__uint_as_float(m << 16) / Q);
  if (__hisinf(hs)) hs = __float2half_rn(65504.f);
  const float sf = __half2float(hs);
  const bool zero = sf == 0.f || sf != sf;
  if (sf == 0.f) hs = __float2half_rn(1.f);
  if (lane_r == 0) (is_v ? c.vs : c.ks)[page * c.scale_stride + prow] = hs;
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  int code[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float(i & 1 ? words[i / 2] & 0xFFFF0000u : words[i / 2] << 16);
    code[i] = zero ? 0 : (int)fminf(fmaxf(rintf(x / sf), -Q), Q);
  }
  if constexpr (KIND == SPEAR_KV_INT8) {
    uint2 o = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.x |= (uint32_t)(code[i] & 0xFF) << (8 * i);
      o.y |= (uint32_t)(code[i + 4] & 0xFF) << (8 * i);
    }
    *reinterpret_cast<uint2*>(dst) = o;
  } else {
    uint32_t o = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) o |= (uint32_t)(code[i] + 8) << (4 * i);
    *reinterpret_cast<uint32_t*>(dst) = o;
  }
}

// The same lanes in the other direction.
template <int KIND, int DIM>
__global__ void __launch_bounds__(256) kv_read_kernel(KvView c, const int* __restrict__ slots, int n,
                                                      __nv_bfloat16* __restrict__ k_out,
                                                      __nv_bfloat16* __restrict__ v_out, WsHeader* hdr) {
  constexpr int LPR = DIM / 8;
  const bool is_v = blockIdx.y != 0;
  const int lane_r = threadIdx.x % LPR;
  const long long row = (long long)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (row >= (long long)n * c.heads) return;
  const int tok = (int)(row / c.heads), head = (int)(row % c.heads);
  const int slot = slots[tok];
  const int page = slot >> c.log_page, off = slot & (c.page_size - 1);
  uint4 o = {0u, 0u, 0u, 0u};
  if (slot >= 0 && page < c.n_pages) {
    const long long prow = (long long)head * c.page_size + off;
    const uint8_t* src = (is_v ? c.v : c.k) + page * c.page_stride + (prow * DIM + lane_r * 8) * kv_bits(KIND) / 8;
    if constexpr (KIND == SPEAR_KV_BF16) {
      o = *reinterpret_cast<const uint4*>(src);
    } else {
      const float s = __half2float((is_v ? c.vs : c.ks)[page * c.scale_stride + prow]);
      float x[8];
      if constexpr (KIND == SPEAR_KV_INT8) {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = s * (float)(int8_t)((i < 4 ? w.x >> (8 * i) : w.y >> (8 * (i - 4))) & 0xFF);
      } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(src);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = s * (float)((int)((w >> (4 * i)) & 0xF) - 8);
      }
      o = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7]));
    }
  } else if (slot >= 0 && lane_r == 0) {
    report_status(hdr, SPEAR_ERR_DEVICE_CHECK);
  }
  *reinterpret_cast<uint4*>((is_v ? v_out : k_out) + row * DIM + lane_r * 8) = o;
}

static int check_tokens(const int* slots, int n, const void* ws, size_t ws_bytes) {
  if (n < 0) return set_error(SPEAR_ERR_INVALID_ARG, "n=%d", n);
  if (!slots || !ws) return set_error(SPEAR_ERR_INVALID_ARG, "NULL pointer");
  if (reinterpret_cast<uintptr_t>(slots) & 3u) return set_error(SPEAR_ERR_ALIGNMENT, "slots must be 4-byte aligned");
  if (!ptr_aligned16(ws)) return set_error(SPEAR_ERR_ALIGNMENT, "unaligned workspace");
  if (ws_bytes < kWsHeaderBytes)
    return set_error(SPEAR_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, kWsHeaderBytes);
  return SPEAR_OK;
}

static int blocks_for(long long rows, int dim) {
  const int per = 256 / (dim / 8);
  return (int)((rows + per - 1) / per);
}

}  // namespace spear

using namespace spear;

extern "C" size_t spear_kv_page_bytes(int kind, int page_size, int n_heads, int head_dim) {
  if (kind < SPEAR_KV_BF16 || kind > SPEAR_KV_INT4) return 0;
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1))) return 0;
  if (n_heads < 1 || n_heads > 1024 || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return 0;
  return (size_t)n_heads * page_size * head_dim * kv_bits(kind) / 8;
}

extern "C" size_t spear_kv_page_scales(int kind, int page_size, int n_heads, int head_dim) {
  if (kind == SPEAR_KV_BF16 || spear_kv_page_bytes(kind, page_size, n_heads, head_dim) == 0) return 0;
  return (size_t)n_heads * page_size;
}

extern "C" int spear_kv_write(const spear_kv_cache* cache, const uint16_t* k, long long ld_k, const uint16_t* v,
                              long long ld_v, const int* slots, int n, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("spear_kv_write");
  clear_error();
  KvView c;
  int rc = check_kv_cache(cache, &c);
  if (rc) return rc;
  if (n == 0) return SPEAR_OK;
  if ((rc = check_tokens(slots, n, ws, ws_bytes))) return rc;
  if (!k || !v) return set_error(SPEAR_ERR_INVALID_ARG, "NULL pointer");
  if (!ptr_aligned16(k) || !ptr_aligned16(v)) return set_error(SPEAR_ERR_ALIGNMENT, "unaligned pointer");
  const long long row = (long long)c.heads * c.dim;
  if (ld_k < row || ld_v < row || ld_k % 8 || ld_v % 8)
    return set_error(SPEAR_ERR_INVALID_ARG, "ld_k=%lld ld_v=%lld: multiples of 8 of at least %lld", ld_k, ld_v, row);
  if ((long long)n * c.heads > (1LL << 33)) return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "n=%d: too many rows", n);
  const dim3 grid(blocks_for((long long)n * c.heads, c.dim), 2);
  for_kind_dim(c.kind, c.dim, [&](auto kc, auto dc) {
    kv_write_kernel<kc.value, dc.value><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        c, reinterpret_cast<const __nv_bfloat16*>(k), ld_k, reinterpret_cast<const __nv_bfloat16*>(v), ld_v, slots, n,
        static_cast<WsHeader*>(ws));
  });
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEAR_OK : set_cuda_error("kv write launch", e);
}

extern "C" int spear_kv_read(const spear_kv_cache* cache, const int* slots, int n, uint16_t* k_out, uint16_t* v_out,
                             void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("spear_kv_read");
  clear_error();
  KvView c;
  int rc = check_kv_cache(cache, &c);
  if (rc) return rc;
  if (n == 0) return SPEAR_OK;
  if ((rc = check_tokens(slots, n, ws, ws_bytes))) return rc;
  if (!k_out || !v_out) return set_error(SPEAR_ERR_INVALID_ARG, "NULL pointer");
  if (!ptr_aligned16(k_out) || !ptr_aligned16(v_out)) return set_error(SPEAR_ERR_ALIGNMENT, "unaligned pointer");
  if ((long long)n * c.heads > (1LL << 33)) return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "n=%d: too many rows", n);
  const dim3 grid(blocks_for((long long)n * c.heads, c.dim), 2);
  for_kind_dim(c.kind, c.dim, [&](auto kc, auto dc) {
    kv_read_kernel<kc.value, dc.value><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        c, slots, n, reinterpret_cast<__nv_bfloat16*>(k_out), reinterpret_cast<__nv_bfloat16*>(v_out),
        static_cast<WsHeader*>(ws));
  });
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEAR_OK : set_cuda_error("kv read launch", e);
}
