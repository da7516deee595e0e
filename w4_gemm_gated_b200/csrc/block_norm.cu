// Norms around a block with its gate and residual scale:
//     u = y * rsqrt(mean(y^2) + eps) * post        (post optional)
//     x_out = a x + b gate u,   h = x_out * rsqrt(mean(x_out^2) + eps) * pre
// in fp32, each output rounded once to bf16.  One CTA per row; the row stays in
// registers between the two reductions, so x and y are read once and x_out
// and h written once: bound by HBM at many rows (8192 x 4096 with a gate per token:
// 336 MB in 53 us, 6.3 TB/s), by the launch and the two block reductions at few
// (one row of 4096: 2.0 us).
#include "kv_cache.cuh"

namespace spear {

struct NormArgs {
  const __nv_bfloat16 *x, *y, *post, *gate, *pre;
  __nv_bfloat16 *x_out, *h;
  long long gate_ld;
  int K;
  float a, b, eps;
};

__device__ __forceinline__ void unpack8(uint4 w, float (&f)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Sum over the block, the same value in every thread; red: one float per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < warps; ++w) s += red[w];
  return s;
}

// V vectors of 8 values per thread: vector j * blockDim.x + threadIdx.x of the
// row.  All of a row's loads go out before the first sum (the weights' too where
// there are registers for them).
template <int V>
__global__ void __launch_bounds__(1024) block_norm_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float red[2][32];
  const long long row = blockIdx.x, base = row * p.K;
  const int nv = p.K / 8;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  uint4 xw[V], yw[V], gw[V], post = none, pre = none;
  after_previous();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    xw[j] = yw[j] = gw[j] = none;
    if (i < nv) {
      if (p.y) yw[j] = *reinterpret_cast<const uint4*>(p.y + base + 8 * i);
      xw[j] = *reinterpret_cast<const uint4*>(p.x + base + 8 * i);
      if (p.gate) gw[j] = *reinterpret_cast<const uint4*>(p.gate + row * p.gate_ld + 8 * i);
      if (V == 1 && p.post) post = *reinterpret_cast<const uint4*>(p.post + 8 * i);
      if (V == 1 && p.pre) pre = *reinterpret_cast<const uint4*>(p.pre + 8 * i);
    }
  }
  float x[V][8];
  if (p.y) {
    float r = 1.f;
    if (p.post) {
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float u[8];
        unpack8(yw[j], u);
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(u[e], u[e], sq);
      }
      r = rsqrtf(block_sum(sq, red[0]) / p.K + p.eps);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = j * blockDim.x + threadIdx.x;
      float u[8], w[8];
      unpack8(yw[j], u);
      if (p.post) {
        if (V > 1 && i < nv) post = *reinterpret_cast<const uint4*>(p.post + 8 * i);
        unpack8(post, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] *= r * w[e];
      }
      if (p.gate) {
        unpack8(gw[j], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] *= w[e];
      }
      unpack8(xw[j], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] = fmaf(p.b, u[e], p.a * w[e]);
      if (p.x_out && i < nv) *reinterpret_cast<uint4*>(p.x_out + base + 8 * i) = pack8(x[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) unpack8(xw[j], x[j]);
  }
  if (!p.h) return;
  float sq = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) sq = fmaf(x[j][e], x[j][e], sq);
  const float r = rsqrtf(block_sum(sq, red[1]) / p.K + p.eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i < nv) {
      if (p.pre) {
        float w[8];
        if (V > 1) pre = *reinterpret_cast<const uint4*>(p.pre + 8 * i);
        unpack8(pre, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] *= r * w[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] *= r;
      }
      *reinterpret_cast<uint4*>(p.h + base + 8 * i) = pack8(x[j]);
    }
  }
}

template <int V>
static cudaError_t launch_norm(const NormArgs& a, int M, cudaStream_t st) {
  const int threads = ((a.K / 8 + V - 1) / V + 31) / 32 * 32;
  return launch_after(block_norm_kernel<V>, dim3(M), threads, 0, st, a);
}

}  // namespace spear

using namespace spear;

extern "C" int spear_block_norm(const uint16_t* x, const uint16_t* y, int M, int K, const uint16_t* post_weight,
                                const uint16_t* gate, long long gate_ld, float residual_scale, float block_scale,
                                const uint16_t* pre_weight, float eps, uint16_t* x_out, uint16_t* h, void* stream) {
  TraceRange trace_("spear_block_norm");
  clear_error();
  if (K < 8 || K > 16384 || K % 8)
    return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "K=%d: must be a multiple of 8, 8 to 16384", K);
  if (M < 0 || M > (1 << 20)) return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "M=%d: must be 0 to 2^20", M);
  if (!(eps >= 0.f)) return set_error(SPEAR_ERR_INVALID_ARG, "eps=%g: must not be negative", eps);
  if (M == 0) return SPEAR_OK;
  if (!x || (!x_out && !h)) return set_error(SPEAR_ERR_INVALID_ARG, "x, and x_out or h, must not be NULL");
  if (!y && (x_out || post_weight || gate))
    return set_error(SPEAR_ERR_INVALID_ARG, "without y there is no x_out, post_weight or gate");
  if (gate && gate_ld != 0 && (gate_ld < K || gate_ld % 8))
    return set_error(SPEAR_ERR_INVALID_ARG, "gate_ld=%lld: 0, or a multiple of 8 of at least K=%d", gate_ld, K);
  for (const void* p : {(const void*)x, (const void*)y, (const void*)post_weight, (const void*)gate,
                        (const void*)pre_weight, (const void*)x_out, (const void*)h})
    if (!ptr_aligned16(p)) return set_error(SPEAR_ERR_ALIGNMENT, "unaligned pointer");
  // outputs may be x or y, element for element, and overlap nothing else
  const uintptr_t rows = (uintptr_t)M * K * 2, one = (uintptr_t)K * 2;
  for (const uint16_t* o : {(const uint16_t*)x_out, (const uint16_t*)h})
    if ((o != x && buffers_meet(o, rows, x, rows)) || (o != y && buffers_meet(o, rows, y, rows)) ||
        buffers_meet(o, rows, post_weight, one) || buffers_meet(o, rows, pre_weight, one) ||
        buffers_meet(o, rows, gate, (uintptr_t)(M - 1) * gate_ld * 2 + one))
      return set_error(SPEAR_ERR_INVALID_ARG, "an output overlaps an input that it is not equal to");
  if (buffers_meet(x_out, rows, h, rows)) return set_error(SPEAR_ERR_INVALID_ARG, "x_out and h overlap");
  auto bf = [](const uint16_t* p) { return reinterpret_cast<const __nv_bfloat16*>(p); };
  const NormArgs a = {bf(x), bf(y), bf(post_weight), bf(gate), bf(pre_weight),
                      reinterpret_cast<__nv_bfloat16*>(x_out), reinterpret_cast<__nv_bfloat16*>(h), gate_ld, K,
                      residual_scale, block_scale, eps};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // One vector per thread while the machine takes all of the call's threads at 1024
  // per SM, where the chain from the loads to the stores counts (4096 wide, one row:
  // 2.0 us against 2.3 with two; 256 rows: 2.9, 3.3); two beyond, whose loads in
  // flight HBM needs (8192 wide, 256 rows: 3.6 us, 5.6 with one; 5120 wide, 8192
  // rows: 51.7, 74.5, with four 52.6)
  const bool one_each = K <= 8192 && (long long)M * K <= 8192LL * device_sm_count();
  const cudaError_t e = one_each ? launch_norm<1>(a, M, st) : launch_norm<2>(a, M, st);
  return e == cudaSuccess ? SPEAR_OK : set_cuda_error("block norm launch", e);
}
