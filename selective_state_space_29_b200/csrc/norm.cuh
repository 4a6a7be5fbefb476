// norm.cuh -- layer norm of rows of channels, and its gradients.
//     mean = sum x / n,  rstd = (sum (x - mean)^2 / n + eps)^-1/2
//     y = (x - mean) rstd weight + bias          (MAMBA_NORM_RMS: mean = 0)
// With xh = (x - mean) rstd and d = dy weight:
//     dx = rstd (d - mean(d) - xh mean(d xh))    (RMS: without mean(d))
//     dweight = sum over rows of dy xh,  dbias = sum over rows of dy
#pragma once

#include "common.cuh"

namespace mamba {

__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (unsigned i = 0; i < blockDim.x / 32; ++i) s += sh[i];
  return s;
}

template <typename TIO>
__global__ void norm_kernel(const TIO* x, const float* weight, const float* bias, TIO* y, float* mean, float* rstd,
                            int64_t channels, float eps, int rms) {
  __shared__ float sh[32];
  const int64_t r = blockIdx.x;
  x += r * channels;
  float s = 0.0f;
  if (!rms) {
    for (int64_t c = threadIdx.x; c < channels; c += blockDim.x) s += to_f32(x[c]);
    s = block_sum(s, sh) / (float)channels;
  }
  float q = 0.0f;
  for (int64_t c = threadIdx.x; c < channels; c += blockDim.x) {
    const float d = to_f32(x[c]) - s;
    q = fmaf(d, d, q);
  }
  const float rs = 1.0f / sqrtf(block_sum(q, sh) / (float)channels + eps);
  if (threadIdx.x == 0) {
    if (mean) mean[r] = s;
    if (rstd) rstd[r] = rs;
  }
  for (int64_t c = threadIdx.x; c < channels; c += blockDim.x) {
    const float v = (to_f32(x[c]) - s) * rs * (weight ? weight[c] : 1.0f);
    y[r * channels + c] = from_f32<TIO>(bias ? v + bias[c] : v);
  }
}

template <typename TIO>
__global__ void norm_input_gradient_kernel(const TIO* dy, const TIO* x, const float* weight, const float* mean,
                                           const float* rstd, TIO* dx, int64_t channels, int rms) {
  __shared__ float sh[32];
  const int64_t r = blockIdx.x;
  const float m = rms ? 0.0f : mean[r], rs = rstd[r];
  x += r * channels;
  dy += r * channels;
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = threadIdx.x; c < channels; c += blockDim.x) {
    const float d = to_f32(dy[c]) * (weight ? weight[c] : 1.0f);
    s1 += d;
    s2 = fmaf(d, (to_f32(x[c]) - m) * rs, s2);
  }
  s1 = rms ? 0.0f : block_sum(s1, sh) / (float)channels;
  s2 = block_sum(s2, sh) / (float)channels;
  for (int64_t c = threadIdx.x; c < channels; c += blockDim.x) {
    const float d = to_f32(dy[c]) * (weight ? weight[c] : 1.0f);
    const float xh = (to_f32(x[c]) - m) * rs;
    dx[r * channels + c] = from_f32<TIO>(rs * ((d - s1) - xh * s2));
  }
}

template <typename TIO>
__global__ void norm_weight_gradient_kernel(const TIO* dy, const TIO* x, const float* mean, const float* rstd,
                                            float* dweight, float* dbias, int64_t rows, int64_t channels, int rms) {
  __shared__ float sw[8][33], sb[8][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float dw = 0.0f, db = 0.0f;
  if (c < channels)
    for (int64_t r = threadIdx.y; r < rows; r += 8) {
      const float d = to_f32(dy[r * channels + c]);
      const float m = rms ? 0.0f : mean[r];
      dw = fmaf(d, (to_f32(x[r * channels + c]) - m) * rstd[r], dw);
      db += d;
    }
  sw[threadIdx.y][threadIdx.x] = dw;
  sb[threadIdx.y][threadIdx.x] = db;
  __syncthreads();
  if (threadIdx.y == 0 && c < channels) {
    for (int i = 1; i < 8; ++i) {
      dw += sw[i][threadIdx.x];
      db += sb[i][threadIdx.x];
    }
    if (dweight) dweight[c] = dw;
    if (dbias) dbias[c] = db;
  }
}

}  // namespace mamba
