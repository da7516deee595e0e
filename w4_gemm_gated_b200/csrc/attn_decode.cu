// Attention of one new token per sequence over the paged cache.
//
// One CTA per (query head, sequence); its warps take tokens in turn, each lane
// holding head_dim / 32 values, with a running maximum and sum of the softmax
// per warp, joined in shared memory at the end.
#include "kv_cache.cuh"

namespace spear {

struct AttnArgs {
  KvView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  const int* table;
  const int* lens;
  long long ld_q, ld_out;
  int ld_table, max_pages, n_seqs, heads, group;
  float scale;
  WsHeader* hdr;
};

template <int KIND, int E>
__device__ __forceinline__ void load_row(const uint8_t* p, float s, int lane, float (&f)[E]) {
  if constexpr (KIND == SPEAR_KV_BF16) {
    const __nv_bfloat16* r = reinterpret_cast<const __nv_bfloat16*>(p) + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = __bfloat162float(r[i]);
  } else if constexpr (KIND == SPEAR_KV_INT8) {
    const int8_t* r = reinterpret_cast<const int8_t*>(p) + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = s * (float)r[i];
  } else {
    const uint8_t* r = p + lane * E / 2;
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = s * (float)((int)((r[i / 2] >> (4 * (i & 1))) & 0xF) - 8);
  }
}

template <int KIND, int DIM>
__global__ void __launch_bounds__(256) attn_kernel(AttnArgs p) {
  constexpr int E = DIM / 32;
  __shared__ float sm_m[8], sm_l[8], sm_acc[8][DIM];
  const int head = blockIdx.x, b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int kvh = head / p.group;
  int len = p.lens[b];
  const long long most = (long long)p.max_pages << p.c.log_page;
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) report_status(p.hdr, SPEAR_ERR_DEVICE_CHECK);
    len = len < 0 ? 0 : (int)most;
  }
  float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(p.q[b * p.ld_q + head * DIM + lane * E + i]) * p.scale;
    acc[i] = 0.f;
  }
  for (int t = warp; t < len; t += 8) {
    const int page = p.table[(long long)b * p.ld_table + (t >> p.c.log_page)];
    float k[E], v[E];
    if ((unsigned)page < (unsigned)p.c.n_pages) {
      const long long prow = (long long)kvh * p.c.page_size + (t & (p.c.page_size - 1));
      const long long at = page * p.c.page_stride + prow * (DIM * kv_bits(KIND) / 8);
      float ks = 1.f, vs = 1.f;
      if constexpr (KIND != SPEAR_KV_BF16) {
        ks = __half2float(p.c.ks[page * p.c.scale_stride + prow]);
        vs = __half2float(p.c.vs[page * p.c.scale_stride + prow]);
      }
      load_row<KIND, E>(p.c.k + at, ks, lane, k);
      load_row<KIND, E>(p.c.v + at, vs, lane, v);
    } else {
      if (lane == 0) report_status(p.hdr, SPEAR_ERR_DEVICE_CHECK);
#pragma unroll
      for (int i = 0; i < E; ++i) k[i] = v[i] = 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    const float m1 = fmaxf(m, s), a = m == -INFINITY ? 0.f : expf(m - m1), e = expf(s - m1);
    m = m1;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * a + e * v[i];
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) sm_acc[warp][lane * E + i] = acc[i];
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < 8; ++w) top = fmaxf(top, sm_m[w]);
  for (int d = threadIdx.x; d < DIM; d += 256) {
    float total = 0.f, o = 0.f;
    for (int w = 0; w < 8; ++w)
      if (sm_m[w] != -INFINITY) {
        const float e = expf(sm_m[w] - top);
        total += e * sm_l[w];
        o += e * sm_acc[w][d];
      }
    p.out[b * p.ld_out + head * DIM + d] = __float2bfloat16_rn(len ? o / total : 0.f);
    if (d == 0 && p.lse) p.lse[(long long)b * p.heads + head] = len ? top + logf(total) : -INFINITY;
  }
}

}  // namespace spear

using namespace spear;

extern "C" size_t spear_attn_workspace_bytes(const spear_kv_cache* cache, int n_q_heads) {
  KvView c;
  if (check_kv_cache(cache, &c) != SPEAR_OK || n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % c.heads) return 0;
  return kWsHeaderBytes;
}

extern "C" int spear_attn_decode(const spear_kv_cache* cache, const uint16_t* q, long long ld_q, int n_seqs,
                                 int n_q_heads, const int* page_table, int max_pages, int ld_table,
                                 const int* seq_lens, float scale, uint16_t* out, long long ld_out, float* lse,
                                 void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("spear_attn_decode");
  clear_error();
  AttnArgs a = {};
  const int rc = check_kv_cache(cache, &a.c);
  if (rc) return rc;
  if (n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % a.c.heads)
    return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "n_q_heads=%d: a multiple of the cache's %d heads, at most 1024",
                     n_q_heads, a.c.heads);
  if (n_seqs < 0 || n_seqs > 4096) return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "n_seqs=%d: must be 0 to 4096", n_seqs);
  if (n_seqs == 0) return SPEAR_OK;
  if (!q || !page_table || !seq_lens || !out || !ws) return set_error(SPEAR_ERR_INVALID_ARG, "NULL pointer");
  if (!(fabsf(scale) < INFINITY)) return set_error(SPEAR_ERR_INVALID_ARG, "scale=%g: must be finite", scale);
  if (q == out) return set_error(SPEAR_ERR_INVALID_ARG, "q and out are the same buffer");
  if (max_pages < 1 || ld_table < max_pages)
    return set_error(SPEAR_ERR_INVALID_ARG, "max_pages=%d ld_table=%d: 1 <= max_pages <= ld_table", max_pages, ld_table);
  if ((long long)max_pages * a.c.page_size > 0x7fffffffLL)
    return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "max_pages=%d: a sequence holds less than 2^31 tokens", max_pages);
  const long long row = (long long)n_q_heads * a.c.dim;
  if (ld_q < row || ld_out < row || ld_q % 8 || ld_out % 8)
    return set_error(SPEAR_ERR_INVALID_ARG, "ld_q=%lld ld_out=%lld: multiples of 8 of at least %lld", ld_q, ld_out, row);
  if (!ptr_aligned16(q) || !ptr_aligned16(out) || !ptr_aligned16(ws))
    return set_error(SPEAR_ERR_ALIGNMENT, "q, out and ws must be 16-byte aligned");
  for (const void* p : {(const void*)page_table, (const void*)seq_lens, (const void*)lse})
    if (reinterpret_cast<uintptr_t>(p) & 3u)
      return set_error(SPEAR_ERR_ALIGNMENT, "page_table, seq_lens and lse must be 4-byte aligned");
  const size_t need = spear_attn_workspace_bytes(cache, n_q_heads);
  if (ws_bytes < need) return set_error(SPEAR_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.table = page_table;
  a.lens = seq_lens;
  a.ld_q = ld_q;
  a.ld_out = ld_out;
  a.ld_table = ld_table;
  a.max_pages = max_pages;
  a.n_seqs = n_seqs;
  a.heads = n_q_heads;
  a.group = n_q_heads / a.c.heads;
  a.scale = scale;
  a.hdr = static_cast<WsHeader*>(ws);
  for_kind_dim(a.c.kind, a.c.dim, [&](auto kc, auto dc) {
    attn_kernel<kc.value, dc.value>
        <<<dim3(n_q_heads, n_seqs), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  });
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEAR_OK : set_cuda_error("attention launch", e);
}
