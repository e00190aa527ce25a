// awq_norm.cuh — the residual update after a block and the RMS norm before the next one.
//
//   t  = y,  or  y / sqrt(mean(y^2) + eps) * w_post      (norm after the block)
//   h  = residual + alpha * gate * t                     (gate and residual scale)
//   x' = h / sqrt(mean(h^2) + eps) * w / s               (norm before the next block, activation scaling)
//
// fp32 throughout, one rounding to fp16 for each of h and x' (the second mean and x' are taken
// from the unrounded h). s is the next linear layer's stored scale (CSDN "02.02 AWQ": activations
// scaled down by s), so x' goes straight into a quantized linear call.
//
// Bound by HBM: 8 bytes per value (10 with a gate per token). One CTA per row; the row stays in
// registers between the two means, so every input is read once, and a thread has read its values of y and
// the residual before it writes h and x there: both may be updated in place. Few rows (a decoding batch) are bound
// by latency and take as many threads as they have 8-value chunks; many rows two chunks per thread,
// four where the norm after the block adds a second reduction and many rows hide it.
// (The division by s is approximate, 2 units of 2^-24, and gives 0 from |s| = 2^126 on, where x' is 0 in fp16
// anyway.)
// Measured: 8192 x 8192 83 us (0.98 of the copy rate; 95 with the IEEE division by s), 90 us with the
// norm after the block (98 with two chunks per thread); 4096 x 8192 with both norms and a gate per token
// 63 us (0.81), 68 without the gate's prefetch, which a few rows of one chunk per thread do not repay
// (300 x 4096 5.3 us, 5.7 with it); 1 x 4096 2.1 us.
#pragma once

#include "awq_common.cuh"

namespace awq {

struct NormArgs {
  const __half* y;
  const __half* residual;   // null: 0
  const __half* gate;       // null: 1; otherwise row m uses gate row m / rows_per_gate
  const __half* post_w;     // null: no norm after the block
  const __half* w;
  const float* s;           // null: 1
  __half* h;                // null: not stored
  __half* x;
  int K, rows_per_gate;
  float alpha, eps;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = half2_bits_to_float2(w[j]);
    f[2 * j] = p.x;
    f[2 * j + 1] = p.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the CTA in a fixed order (lanes by halving, then the warps' sums by every warp alike).
__device__ __forceinline__ float block_sum(float v, float* s_part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int lane = threadIdx.x & 31;
  if (lane == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < static_cast<int>(blockDim.x >> 5) ? s_part[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Threads that a row takes with VPT 8-value chunks per thread: at most 768 with two chunks, so that two
// CTAs fit an SM's registers.
constexpr int norm_max_threads(int vpt) { return vpt == 2 ? 768 : 1024; }

template <int VPT>
__global__ void __launch_bounds__(norm_max_threads(VPT)) awq_residual_norm_kernel(const NormArgs a) {
  pdl_enter_early();
  __shared__ float s_part[2][32];
  const size_t row = blockIdx.x;
  const int chunks = a.K / 8, tid = threadIdx.x, nthr = blockDim.x;
  const float inv_k = 1.0f / static_cast<float>(a.K);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const size_t base = row * a.K;
  auto inside = [&](int c) { return AWQ_CHECK(c >= 0 && 8 * c + 8 <= a.K && row < gridDim.x); };
  uint4 yv[VPT], rv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * nthr;
    yv[i] = c < chunks && inside(c) ? ld_stream_v4(a.y + base + c * 8) : zero;
    rv[i] = c < chunks && a.residual != nullptr && inside(c) ? ld_stream_v4(a.residual + base + c * 8) : zero;
  }
  float rstd = 1.0f;
  if (a.post_w != nullptr) {
    if (VPT > 1 && a.gate != nullptr) {        // the gate is on its way into L2 during the reduction
      const __half* g = a.gate + row / a.rows_per_gate * a.K;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * nthr;
        if (c < chunks && (c & 7) == 0 && inside(c)) asm volatile("prefetch.global.L2 [%0];" ::"l"(g + c * 8));
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
      unpack8(yv[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
    }
    rstd = __frsqrt_rn(fmaf(block_sum(sum, s_part[0]), inv_k, a.eps));
  }
  float h[VPT][8];
  float sum = 0.0f;
  const __half* gate = a.gate == nullptr ? nullptr : a.gate + row / a.rows_per_gate * a.K;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * nthr;
    float r[8];
    unpack8(yv[i], h[i]);
    unpack8(rv[i], r);
    if (a.post_w != nullptr && c < chunks && inside(c)) {
      float w[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(a.post_w + c * 8)), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * rstd * w[j];
    }
    if (gate != nullptr && c < chunks && inside(c)) {
      float g[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(gate + c * 8)), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] *= g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[i][j] = fmaf(a.alpha, h[i][j], r[j]);
      sum = fmaf(h[i][j], h[i][j], sum);
    }
    if (a.h != nullptr && c < chunks && inside(c)) *reinterpret_cast<uint4*>(a.h + base + c * 8) = pack8(h[i]);
  }
  rstd = __frsqrt_rn(fmaf(block_sum(sum, s_part[1]), inv_k, a.eps));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * nthr;
    if (c >= chunks || !inside(c)) continue;
    float w[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(a.w + c * 8)), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= h[i][j] * rstd;
    if (a.s != nullptr) {
      const float4 s0 = __ldg(reinterpret_cast<const float4*>(a.s + c * 8));
      const float4 s1 = __ldg(reinterpret_cast<const float4*>(a.s + c * 8 + 4));
      const float sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __fdividef(w[j], sc[j]);   // 2 units of 2^-24: far below the fp16 step
    }
    *reinterpret_cast<uint4*>(a.x + base + c * 8) = pack8(w);
  }
}

}  // namespace awq
