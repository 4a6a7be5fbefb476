// norm.cuh -- layer norm of rows of channels, and its gradients.
//     mean = sum x / n,  rstd = (sum (x - mean)^2 / n + eps)^-1/2
//     y = (x - mean) rstd weight + bias          (MAMBA_NORM_RMS: mean = 0)
// With xh = (x - mean) rstd and d = dy weight:
//     dx = rstd (d - mean(d) - xh mean(d xh))    (RMS: without mean(d))
//     dweight = sum over rows of dy xh,  dbias = sum over rows of dy
//
// Both directions are bound by HBM: 4 bytes an element forward and 6 backward
// (bf16), each read once into registers and held there for the sums and the
// outputs.  A row is held by LR lanes, a power of two from 4 to 512, each with
// VPL vectors of E elements (16 bytes, or one element where rows are not
// 16-byte aligned); sums go by shuffles, and through shared memory where a row
// has several warps.
#pragma once

#include "common.cuh"

namespace mamba {

// E elements of TIO, as loaded
template <typename TIO, int E>
struct NormVec {
  static_assert(E == 1 || E * sizeof(TIO) == 16, "one element or 16 bytes");
  uint32_t w[E == 1 ? 1 : 4];
  __device__ __forceinline__ void load(const TIO* p) {
    if constexpr (E == 1) {
      if constexpr (sizeof(TIO) == 4) w[0] = __float_as_uint(__ldg(p));
      else w[0] = (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16;
    } else {
      // read once: kept out of L1, which holds weight and bias
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (E == 1 ? 1 : 4); ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (E == 1 || sizeof(TIO) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};

template <typename TIO, int E>
__device__ __forceinline__ void norm_store(TIO* p, const float (&v)[E]) {
  if constexpr (E == 1) {
    *p = from_f32<TIO>(v[0]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(TIO) == 4) w[i] = __float_as_uint(v[i]);
      else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// E float32 parameters (weight, bias), or `none` where there are none
template <int E>
__device__ __forceinline__ void norm_param(const float* p, int64_t at, float none, bool wide, float (&v)[E]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = none;
  } else if (E >= 4 && wide) {
#pragma unroll
    for (int i = 0; i + 3 < E; i += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p + at + i));
      v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = __ldg(p + at + i);
  }
}

// Sums of K values over the LR lanes of a row, in every lane.  `sh` has K
// floats per warp; rows of several warps meet at barrier `bar` (their lanes
// only), which also closes the previous use of the other half of `sh`.
template <int K>
__device__ __forceinline__ void norm_row_sum(float (&v)[K], int lr, float* sh, int bar) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    for (int o = 1; o < lr && o < 32; o <<= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  if (lr > 32) {
    const int warps = lr >> 5, warp = threadIdx.x >> 5, first = warp & ~(warps - 1);
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) sh[warp * K + k] = v[k];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(lr) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.0f;
    for (int w = 0; w < warps; ++w) {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += sh[(first + w) * K + k];
    }
  }
}

struct NormArgs {
  const void* x;
  const void* dy;
  const float* weight;
  const float* bias;
  void* y;             // dx in the backward
  float* mean;
  float* rstd;
  const float* mean_in;
  const float* rstd_in;
  float* part;         // [ctas][2][channels]: sums of dy xh, dy
  float* dweight;
  float* dbias;
  int64_t rows;
  int channels;
  int lr_log2;
  int wide;            // weight and bias 16-byte aligned
  int rms;
  float eps;
};

constexpr int kNormMaxThreads = 512;

template <typename TIO, int E, int VPL>
__global__ void __launch_bounds__(kNormMaxThreads) norm_kernel(const NormArgs p) {
  __shared__ float sh[2][kNormMaxThreads / 32];
  const int lr = 1 << p.lr_log2, slot = threadIdx.x >> p.lr_log2, lane = threadIdx.x & (lr - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> p.lr_log2) + slot;
  const bool live = row < p.rows;
  const TIO* x = static_cast<const TIO*>(p.x) + row * p.channels;
  const float n = (float)p.channels;
  griddep_launch_dependents();
  griddep_wait();

  NormVec<TIO, E> v[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int c = (lane + (j << p.lr_log2)) * E;
    if (live && c < p.channels) v[j].load(x + c);
    else v[j].zero();
  }
  float mean = 0.0f;
  if (!p.rms) {
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < VPL; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] += v[j].get(e);
    norm_row_sum<1>(s, lr, sh[0], 1 + slot);
    mean = s[0] / n;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    if ((lane + (j << p.lr_log2)) * E < p.channels) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = v[j].get(e) - mean;
        q[0] = fmaf(d, d, q[0]);
      }
    }
  }
  norm_row_sum<1>(q, lr, sh[1], 1 + slot);
  const float rstd = 1.0f / sqrtf(q[0] / n + p.eps);
  if (!live) return;
  if (lane == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  TIO* y = static_cast<TIO*>(p.y) + row * p.channels;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int c = (lane + (j << p.lr_log2)) * E;
    if (c < p.channels) {
      float w[E], b[E], o[E];
      norm_param<E>(p.weight, c, 1.0f, p.wide, w);
      norm_param<E>(p.bias, c, 0.0f, p.wide, b);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf((v[j].get(e) - mean) * rstd, w[e], b[e]);
      norm_store<TIO, E>(y + c, o);
    }
  }
}

// A CTA per SM walks rows; its lanes keep their channels' weight and sums of
// dy xh and dy in registers, and hold the next row while they work on this
// one.  The CTA's rows' sums are joined in shared memory and written to `part`.
template <typename TIO, int E, int VPL>
__global__ void __launch_bounds__(kNormMaxThreads) norm_backward_kernel(const NormArgs p) {
  extern __shared__ float dyn[];
  __shared__ float sh[2][2 * kNormMaxThreads / 32];
  const int lr = 1 << p.lr_log2, slot = threadIdx.x >> p.lr_log2, lane = threadIdx.x & (lr - 1);
  const int slots = blockDim.x >> p.lr_log2;
  const float n = (float)p.channels;
  griddep_launch_dependents();
  griddep_wait();

  float w[VPL][E], dw[VPL][E], db[VPL][E];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int c = (lane + (j << p.lr_log2)) * E;
    if (c < p.channels) norm_param<E>(p.weight, c, 1.0f, p.wide, w[j]);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[j][e] = db[j][e] = 0.0f;
  }
  NormVec<TIO, E> x[VPL], g[VPL];
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t row) {
    const bool live = row < p.rows;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = (lane + (j << p.lr_log2)) * E;
      if (live && c < p.channels) {
        x[j].load(static_cast<const TIO*>(p.x) + row * p.channels + c);
        g[j].load(static_cast<const TIO*>(p.dy) + row * p.channels + c);
      } else {
        x[j].zero();
        g[j].zero();
      }
    }
    mean = live && !p.rms ? __ldg(p.mean_in + row) : 0.0f;
    rstd = live ? __ldg(p.rstd_in + row) : 0.0f;
  };
  const int64_t step = (int64_t)gridDim.x * slots;
  int64_t row = (int64_t)blockIdx.x * slots + slot;
  load(row);
  // every slot takes the same number of rounds, so that whole warps stay together
  const int64_t rounds = (p.rows - (int64_t)blockIdx.x * slots + step - 1) / step;
  for (int64_t it = 0; it < rounds; ++it, row += step) {
    const NormVec<TIO, E>*px = x, *pg = g;
    NormVec<TIO, E> cx[VPL], cg[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      cx[j] = px[j];
      cg[j] = pg[j];
    }
    const float m = mean, r = rstd;
    const bool live = row < p.rows;
    load(it + 1 < rounds ? row + step : p.rows);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if ((lane + (j << p.lr_log2)) * E < p.channels) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float gy = cg[j].get(e), xh = (cx[j].get(e) - m) * r, d = gy * w[j][e];
          s[0] += d;
          s[1] = fmaf(d, xh, s[1]);
          dw[j][e] = fmaf(gy, xh, dw[j][e]);
          db[j][e] += gy;
        }
      }
    }
    norm_row_sum<2>(s, lr, sh[it & 1], 1 + slot);
    const float s1 = p.rms ? 0.0f : s[0] / n, s2 = s[1] / n;
    if (live) {
      TIO* dx = static_cast<TIO*>(p.y) + row * p.channels;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int c = (lane + (j << p.lr_log2)) * E;
        if (c < p.channels) {
          float o[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float xh = (cx[j].get(e) - m) * r;
            o[e] = r * (fmaf(cg[j].get(e), w[j][e], -s1) - xh * s2);
          }
          norm_store<TIO, E>(dx + c, o);
        }
      }
    }
  }
  if (p.part == nullptr) return;
  // the slots' sums, one after the other in a fixed order
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.channels;
  const int held = lr * VPL * E;  // channels a slot holds
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VPL; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e)
        dyn[slot * held + (lane + (j << p.lr_log2)) * E + e] = k == 0 ? dw[j][e] : db[j][e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.channels; c += blockDim.x) {
      float t = 0.0f;
      for (int s = 0; s < slots; ++s) t += dyn[s * held + c];
      part[k * p.channels + c] = t;
    }
  }
}

// dweight and dbias from the CTAs' sums: 32 channels by 32 runs of CTAs, joined
// in order.
__global__ void __launch_bounds__(1024) norm_join_kernel(const NormArgs p, int ctas) {
  __shared__ float sh[32][33];
  const int k = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  float* out = k == 0 ? p.dweight : p.dbias;
  griddep_launch_dependents();
  griddep_wait();
  if (out == nullptr) return;
  float t = 0.0f;
  if (c < p.channels)
    for (int i = threadIdx.y; i < ctas; i += 32) t += p.part[((int64_t)i * 2 + k) * p.channels + c];
  sh[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  t = sh[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < p.channels) out[blockIdx.x * 32 + threadIdx.y] = t;
}

}  // namespace mamba
