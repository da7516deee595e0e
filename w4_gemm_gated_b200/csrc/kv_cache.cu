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

// Rows of the calls: token-major, DIM / 16 lanes per row, each with the two
// chunks of 8 values that lie DIM / 2 apart (so that every load and store of a
// warp is of whole sectors).  At large sizes both calls are as near the issue
// rate as HBM, so what a row costs beside its values is spread over 16 of them (8
// per lane took 1.2 times as long to read back, 1.6 times to write).
// 29,300 tokens of 8 int8 heads are read back in 31.7 us, 87 % of what a copy of as
// many bytes reaches, 7,200 written in 9.9 us, 68 % (of bf16 heads 96 and 84 %).
constexpr int kThreads = 256;

// Token and head of a row.  magic = floor(2^32 / heads): the product's high half is
// the quotient or one less.
__device__ __forceinline__ void split_row(unsigned row, unsigned heads, unsigned magic, unsigned& tok, unsigned& head) {
  tok = heads == 1 ? row : __umulhi(row, magic);
  head = row - tok * heads;
  if (head >= heads) ++tok, head -= heads;
}

// Two fp32 values in one register pair, and operations on both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 8 bf16 values -> codes c = clamp(rint(x / s), -Q, Q) of the IEEE quotient, as bytes.
//
// x has 8 significant bits and s 11, so a quotient of at most 128 that is no tie
// (k + 1/2) is at least 1 / (2 * 2047) = 2.4e-4 away from one; x * (1 / s), with a
// reciprocal of up to 2 ulp, is within 2^-22 * 128 = 3.1e-5 of it.  Rounded once to a
// multiple of 2^-13 (with 1.5 * 2^10 added, where that is the spacing; off by 6.1e-5
// more at most), a tie becomes the tie exactly and nothing else does, and rounding
// that to an integer (with 1.5 * 2^23 in the other's place, whose low byte then
// holds it) is the definition's.
// clamp: the row's scale was cut or is below fp16's normal range, so that
// quotients pass Q (elsewhere they stay under Q (1 + 2^-11), which rounds to Q).
template <int Q>
__device__ __forceinline__ void quantize8(const uint4& in, float inv, bool clamp, uint32_t& lo, uint32_t& hi) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  constexpr float kGrid = 1536.f, kWhole = 12582912.f;
  const uint64_t inv2 = pair(inv, inv), grid = pair(kGrid, kGrid), whole = pair(kWhole - kGrid, kWhole - kGrid);
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t t = fma2(pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), inv2, grid);
    float a, b;
    if (clamp) {
      unpair(t, a, b);
      t = pair(fminf(fmaxf(a, kGrid - Q), kGrid + Q), fminf(fmaxf(b, kGrid - Q), kGrid + Q));
    }
    unpair(add2(t, whole), a, b);
    y[2 * i] = __float_as_uint(a);
    y[2 * i + 1] = __float_as_uint(b);
  }
  lo = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
  hi = __byte_perm(__byte_perm(y[4], y[5], 0x0040), __byte_perm(y[6], y[7], 0x0040), 0x5410);
}

// N bytes of a row as words.
template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t* src, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(src);
  }
}

// STEP rows per thread, whose loads are in flight together.
template <int KIND, int DIM, int STEP>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const __grid_constant__ KvView c,
                                                            const __nv_bfloat16* k, long long ld_k,
                                                            const __nv_bfloat16* v, long long ld_v,
                                                            const int* slots, unsigned rows,
                                                            unsigned magic, WsHeader* hdr) {
  constexpr int LPR = DIM / 16, RPS = kThreads / LPR, BYTES = kv_bits(KIND);  // bytes of 8 values
  const bool is_v = blockIdx.y != 0;
  const int lane_r = threadIdx.x % LPR;
  const unsigned row0 = blockIdx.x * (STEP * RPS) + threadIdx.x / LPR;
  after_previous();
  int slot[STEP];
  unsigned head[STEP];
  uint4 in[STEP][2];
#pragma unroll
  for (int u = 0; u < STEP; ++u) {
    const unsigned row = row0 + u * RPS;
    unsigned tok;
    split_row(row, c.heads, magic, tok, head[u]);
    slot[u] = -1;
    in[u][0] = in[u][1] = make_uint4(0u, 0u, 0u, 0u);
    if (row < rows) {
      slot[u] = slots[tok];
      const __nv_bfloat16* x = (is_v ? v : k) + tok * (is_v ? ld_v : ld_k) + head[u] * DIM + lane_r * 8;
      in[u][0] = *reinterpret_cast<const uint4*>(x);
      in[u][1] = *reinterpret_cast<const uint4*>(x + DIM / 2);
    }
  }
#pragma unroll
  for (int u = 0; u < STEP; ++u) {
    const int page = slot[u] >> c.log_page;
    const bool live = slot[u] >= 0 && page < c.n_pages && SPEAR_DCHECK(head[u] < (unsigned)c.heads, hdr);
    if (slot[u] >= 0 && !live && lane_r == 0) report_status(hdr, SPEAR_ERR_DEVICE_CHECK);
    const int prow = (head[u] << c.log_page) + (slot[u] & (c.page_size - 1));  // row inside the page
    uint8_t* dst = (is_v ? c.v : c.k) + (page_at(live ? page : 0, c.page_step) << 4) +
                   (long long)prow * (DIM / 8 * BYTES) + lane_r * BYTES;
    if constexpr (KIND == SPEAR_KV_BF16) {
      if (live) {
        *reinterpret_cast<uint4*>(dst) = in[u][0];
        *reinterpret_cast<uint4*>(dst + DIM / 16 * BYTES) = in[u][1];
      }
    } else {
      constexpr int Q = KIND == SPEAR_KV_INT8 ? 127 : 7;
      // max of the magnitudes as 16-bit patterns: a NaN's pattern is above infinity's
      uint32_t m2 = 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        m2 = absmax2(absmax2(absmax2(absmax2(m2, in[u][h].x), in[u][h].y), in[u][h].z), in[u][h].w);
      uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
      for (int d = LPR / 2; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d, LPR));
      __half hs = __float2half_rn(__uint_as_float(m << 16) / (float)Q);
      if (__hisinf(hs)) hs = __float2half_rn(65504.f);
      float sf = __half2float(hs);
      const bool zero = sf == 0.f || sf != sf;  // codes 0: nothing there, or a NaN that the scale keeps
      if (sf == 0.f) hs = __float2half_rn(1.f);
      if (zero) sf = 1.f;
      const float inv = __fdividef(1.f, sf);
      const bool clamp = __any_sync(0xFFFFFFFFu, sf < 6.103515625e-5f || sf >= 65504.f || zero);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t lo, hi;
        quantize8<Q>(in[u][h], inv, clamp, lo, hi);
        if (zero) lo = hi = 0u;
        uint8_t* d = dst + h * (DIM / 16 * BYTES);
        if constexpr (KIND == SPEAR_KV_INT8) {
          if (live) *reinterpret_cast<uint2*>(d) = make_uint2(lo, hi);
        } else {
          // codes + 8 in the low half of each byte; neighbours into one byte
          lo = __vadd4(lo, 0x08080808u), hi = __vadd4(hi, 0x08080808u);
          lo = (lo | lo >> 4) & 0x00FF00FFu, hi = (hi | hi >> 4) & 0x00FF00FFu;
          if (live) *reinterpret_cast<uint32_t*>(d) = __byte_perm(lo, hi, 0x6420);
        }
      }
      if (live && lane_r == 0) (is_v ? c.vs : c.ks)[(page_at(page, c.scale_step) << 3) + prow] = hs;
    }
  }
}

// As above, back.
template <int KIND, int DIM, int STEP>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvView c,
                                                           const int* slots, unsigned rows,
                                                           unsigned magic, __nv_bfloat16* k_out,
                                                           __nv_bfloat16* v_out, WsHeader* hdr) {
  constexpr int LPR = DIM / 16, RPS = kThreads / LPR, BYTES = kv_bits(KIND), WORDS = BYTES / 4;
  const bool is_v = blockIdx.y != 0;
  const int lane_r = threadIdx.x % LPR;
  const unsigned row0 = blockIdx.x * (STEP * RPS);
  after_previous();
  const uint8_t* codes = (is_v ? c.v : c.k) + lane_r * BYTES;
  const __half* scales = is_v ? c.vs : c.ks;
  uint32_t in[STEP][2][WORDS];
  float scale[STEP];
  bool live[STEP];
#pragma unroll
  for (int u = 0; u < STEP; ++u) {
    const int r = u * RPS + threadIdx.x / LPR;
    live[u] = false;
    if (row0 + r < rows) {
      unsigned tok, head;
      split_row(row0 + r, c.heads, magic, tok, head);
      const int slot = slots[tok];
      const int page = slot >> c.log_page;
      live[u] = slot >= 0 && page < c.n_pages && SPEAR_DCHECK(head < (unsigned)c.heads, hdr);
      if (live[u]) {
        const int prow = (head << c.log_page) + (slot & (c.page_size - 1));
        const uint8_t* src = codes + (page_at(page, c.page_step) << 4) + (long long)prow * (DIM / 8 * BYTES);
        load_words(src, in[u][0]);
        load_words(src + DIM / 16 * BYTES, in[u][1]);
        if constexpr (KIND != SPEAR_KV_BF16) scale[u] = __half2float(scales[(page_at(page, c.scale_step) << 3) + prow]);
      } else if (slot >= 0 && lane_r == 0) {
        report_status(hdr, SPEAR_ERR_DEVICE_CHECK);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < STEP; ++u) {
    const unsigned row = row0 + u * RPS + threadIdx.x / LPR;
    if (row >= rows) continue;
    __nv_bfloat16* out = (is_v ? v_out : k_out) + (long long)row * DIM + lane_r * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 o = make_uint4(0u, 0u, 0u, 0u);
      if (live[u]) {
        if constexpr (KIND == SPEAR_KV_BF16) {
          o = make_uint4(in[u][h][0], in[u][h][1], in[u][h][2], in[u][h][3]);
        } else {
          // a byte b in the low bits of 2^23 is 2^23 + b; the codes' offsets (128,
          // 8) come off with it, exactly, and the product with the scale is exact
          // too (8 bits by 11), so that the one rounding is to bf16
          uint32_t b[2];
          if constexpr (KIND == SPEAR_KV_INT8) {
            b[0] = in[u][h][0] ^ 0x80808080u, b[1] = in[u][h][1] ^ 0x80808080u;
          } else {  // values 2i in b[0], 2i + 1 in b[1]
            b[0] = in[u][h][0] & 0x0F0F0F0Fu, b[1] = in[u][h][0] >> 4 & 0x0F0F0F0Fu;
          }
          constexpr float kOff = KIND == SPEAR_KV_INT8 ? -8388736.f : -8388616.f;
          const uint64_t off = pair(kOff, kOff), s2 = pair(scale[u], scale[u]);
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x0 = KIND == SPEAR_KV_INT8 ? __byte_perm(b[i / 2], 0x4B000000u, 0x7440 + 2 * (i & 1))
                                                      : __byte_perm(b[0], 0x4B000000u, 0x7440 + i);
            const uint32_t x1 = KIND == SPEAR_KV_INT8 ? __byte_perm(b[i / 2], 0x4B000000u, 0x7440 + 2 * (i & 1) + 1)
                                                      : __byte_perm(b[1], 0x4B000000u, 0x7440 + i);
            float a, z;
            unpair(mul2(add2(pair(__uint_as_float(x0), __uint_as_float(x1)), off), s2), a, z);
            w[i] = pack_bf16x2(a, z);
          }
          o = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      *reinterpret_cast<uint4*>(out + h * (DIM / 2)) = o;
    }
  }
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

// Whether two of a cache's arrays of pages share bytes.  Those whose pages lie as far
// apart may lie beside one another in larger pages; of others nothing is said where
// their ranges meet.
static bool pages_meet(const void* a, long long step_a, long long bytes_a, const void* b, long long step_b,
                       long long bytes_b, int n_pages) {
  if (!buffers_meet(a, (n_pages - 1) * step_a + bytes_a, b, (n_pages - 1) * step_b + bytes_b)) return false;
  if (n_pages == 1) return true;
  if (step_a != step_b) return false;
  const long long apart = (long long)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const long long column = (apart % step_a + step_a) % step_a;
  return column < bytes_a || column + bytes_b > step_a;
}

static bool parts_meet(const KvView& c) {
  const long long codes = (long long)c.heads * c.dim * kv_bits(c.kind) / 8 << c.log_page;
  const long long scales = (long long)c.heads * 2 << c.log_page;
  const void* part[4] = {c.k, c.v, c.ks, c.vs};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (pages_meet(part[i], i < 2 ? c.page_stride : c.scale_stride * 2, i < 2 ? codes : scales, part[j],
                     j < 2 ? c.page_stride : c.scale_stride * 2, j < 2 ? codes : scales, c.n_pages))
        return true;
  return false;
}

static int blocks_for(long long rows, int dim, int step) {
  const int per = step * kThreads / (dim / 16);
  return (int)((rows + per - 1) / per);
}

// Rows per thread: one while the blocks are few, where only a
// call's latency counts (330 tokens of 8 int8 heads: 1.85 us, 2.3 with two), two
// beyond (29,300: 31.7 us, 33.4 with one; 7,200 written: 9.9 us, 10.3 with one).
static int step_for(long long rows, int dim) { return blocks_for(rows, dim, 1) <= 4 * device_sm_count() ? 1 : 2; }

static unsigned magic_for(int heads) { return (unsigned)((1ull << 32) / heads); }

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
  if (parts_meet(c)) return set_error(SPEAR_ERR_INVALID_ARG, "the cache's k, v and scales overlap");
  if ((long long)n * c.heads > (1LL << 31)) return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "n=%d: too many rows", n);
  const unsigned rows = (unsigned)n * c.heads;
  const int step = step_for(rows, c.dim);
  const dim3 grid(blocks_for(rows, c.dim, step), 2);
  cudaError_t e = cudaErrorInvalidValue;
  for_kind_dim(c.kind, c.dim, [&](auto kc, auto dc) {
    auto* f = step == 1 ? kv_write_kernel<kc.value, dc.value, 1> : kv_write_kernel<kc.value, dc.value, 2>;
    e = launch_after(f, grid, kThreads, 0, static_cast<cudaStream_t>(stream), c,
                     reinterpret_cast<const __nv_bfloat16*>(k), ld_k, reinterpret_cast<const __nv_bfloat16*>(v), ld_v,
                     slots, rows, magic_for(c.heads), static_cast<WsHeader*>(ws));
  });
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
  if ((long long)n * c.heads > (1LL << 31)) return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "n=%d: too many rows", n);
  const uintptr_t bytes = (uintptr_t)n * c.heads * c.dim * 2;
  if (buffers_meet(k_out, bytes, v_out, bytes)) return set_error(SPEAR_ERR_INVALID_ARG, "k_out and v_out overlap");
  const unsigned rows = (unsigned)n * c.heads;
  const int step = step_for(rows, c.dim);
  const dim3 grid(blocks_for(rows, c.dim, step), 2);
  cudaError_t e = cudaErrorInvalidValue;
  for_kind_dim(c.kind, c.dim, [&](auto kc, auto dc) {
    auto* f = step == 1 ? kv_read_kernel<kc.value, dc.value, 1> : kv_read_kernel<kc.value, dc.value, 2>;
    e = launch_after(f, grid, kThreads, 0, static_cast<cudaStream_t>(stream), c, slots, rows, magic_for(c.heads),
                     reinterpret_cast<__nv_bfloat16*>(k_out), reinterpret_cast<__nv_bfloat16*>(v_out),
                     static_cast<WsHeader*>(ws));
  });
  return e == cudaSuccess ? SPEAR_OK : set_cuda_error("kv read launch", e);
}
