// gated.cuh -- the gated linear recurrence: one state per channel, its decay
// given per token (no B or C).  Per (batch b, channel c), with g the gate:
//     a_t = 1 / (1 + exp(-g_t))   or, MAMBA_GATE_LOG,  a_t = exp(g_t)
//     w_t = 1                     or, MAMBA_GATE_CONVEX, w_t = 1 - a_t
//     h_t = a_t h_{t-1} + w_t x_t,   y_t = h_t
// and its gradients, from the adjoint lam of h:
//     lam_t = dy_t + a_{t+1} lam_{t+1}
//     dx_t  = w_t lam_t
//     dg_t  = lam_t (h_{t-1} [- x_t if convex]) da/dg,  da/dg = a (1 - a) or a
//     dh0   = a_0 lam_0
//
// Time is cut into blocks of 256 tokens.  A block is the map
// h -> P h + H of its entering state (P the product of its gates, H its end
// state from zero); composing the maps gives the state that enters every
// block, from which the block's outputs follow.  The adjoint is the same
// with time reversed.
#pragma once

#include "common.cuh"

namespace mamba {

constexpr int kGatedBlock = MAMBA_GATED_SCAN_BLOCK;

// a and 1 - a of a gate.  1 - a has no cancellation: for the sigmoid it is
// e a with e = exp(-g) while a >= 1/2.  FAST (bf16 data, whose outputs carry
// 2^-9): hardware exp2 and reciprocal, about 2^-22 off; else the CUDA library's.
template <bool LOG, bool FAST>
__device__ __forceinline__ void gate_decay(float g, float& a, float& one_less) {
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (LOG) {
    if constexpr (FAST) {
      a = ex2_approx(g * kLog2e);
      // exp(g) - 1 = g (1 + g/2 (1 + g/3 (...))): the first term left out is below 2^-20 of it
      float p = fmaf(g, 1.0f / 720.0f, 1.0f / 120.0f);
      p = fmaf(p, g, 1.0f / 24.0f);
      p = fmaf(p, g, 1.0f / 6.0f);
      p = fmaf(p, g, 0.5f);
      p = fmaf(p, g, 1.0f);
      one_less = fabsf(g) < 0.3f ? -g * p : 1.0f - a;
    } else {
      const float m = expm1f(g);
      a = expf(g);
      one_less = -m;
    }
  } else {
    const float e = FAST ? ex2_approx(-g * kLog2e) : expf(-g);
    a = FAST ? __fdividef(1.0f, 1.0f + e) : 1.0f / (1.0f + e);
    if (!(e < 3.0e38f)) a = e == e ? 0.0f : e;
    one_less = e > 1.0f ? 1.0f - a : e * a;
  }
}

struct GatedArgs {
  const void* x;
  const void* gate;
  const void* dy;
  const float* h0;       // [batch][channels] or NULL
  const float* dh;       // gradient of the final state, or NULL
  void* y;               // NULL: only checkpoints / final state
  float* final_state;    // or NULL
  float* ckpt;           // [batch][blocks][channels]: state entering each block, or NULL
  void* dx;
  void* dgate;
  float* dh0;
  float2* agg;           // [batch][blocks][channels] (P, H)
  float* enter;          // [batch][blocks][channels]: adjoint entering a block from the right
  float* hs;             // backward: [batch][len][channels] states before each token
  int64_t len, channels, blocks, batch;
  unsigned ctiles;       // ceil(channels / threads)
};

// (P, H) of every block.  REVERSE: of the adjoint; the block's map takes
// a_{t+1} lam_{t+1} for its last token t.
template <typename TIO, bool LOG, bool CONVEX, bool REVERSE>
__global__ void gated_block_kernel(const GatedArgs p) {
  const int64_t c = (int64_t)(blockIdx.x % p.ctiles) * blockDim.x + threadIdx.x;
  const int64_t kb = blockIdx.x / p.ctiles, k = kb % p.blocks, b = kb / p.blocks;
  if (c >= p.channels) return;
  const int64_t t0 = k * kGatedBlock, t1 = min(p.len, t0 + kGatedBlock);
  const TIO* g = static_cast<const TIO*>(p.gate) + b * p.len * p.channels + c;
  const TIO* v = static_cast<const TIO*>(REVERSE ? p.dy : p.x) + b * p.len * p.channels + c;
  float P = 1.0f, H = 0.0f;
  for (int64_t i = 0; i < t1 - t0; ++i) {
    const int64_t t = REVERSE ? t1 - 1 - i : t0 + i;
    float a, w;
    gate_decay<LOG, sizeof(TIO) == 2>(to_f32(g[t * p.channels]), a, w);
    const float in = to_f32(v[t * p.channels]);
    if (REVERSE) {
      H = a * (H + in);
    } else {
      H = fmaf(a, H, CONVEX ? w * in : in);
    }
    P *= a;
  }
  p.agg[(b * p.blocks + k) * p.channels + c] = make_float2(P, H);
}

// states entering every block (REVERSE: a_{t+1} lam_{t+1} entering from the right)
template <bool REVERSE>
__global__ void gated_carry_kernel(const GatedArgs p) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= p.batch * p.channels) return;
  const int64_t b = i / p.channels, c = i % p.channels;
  const float* first = REVERSE ? p.dh : p.h0;
  float* out = REVERSE ? p.enter : p.ckpt;
  float h = first ? first[i] : 0.0f;
  for (int64_t j = 0; j < p.blocks; ++j) {
    const int64_t at = (b * p.blocks + (REVERSE ? p.blocks - 1 - j : j)) * p.channels + c;
    const float2 ph = p.agg[at];
    out[at] = h;
    h = fmaf(ph.x, h, ph.y);
  }
  if (REVERSE) {
    if (p.dh0) p.dh0[i] = h;
  } else if (p.final_state) {
    p.final_state[i] = h;
  }
}

template <typename TIO, bool LOG, bool CONVEX>
__global__ void gated_output_kernel(const GatedArgs p) {
  const int64_t c = (int64_t)(blockIdx.x % p.ctiles) * blockDim.x + threadIdx.x;
  const int64_t kb = blockIdx.x / p.ctiles, k = kb % p.blocks, b = kb / p.blocks;
  if (c >= p.channels) return;
  const int64_t t0 = k * kGatedBlock, t1 = min(p.len, t0 + kGatedBlock);
  const int64_t base = b * p.len * p.channels + c;
  const TIO* g = static_cast<const TIO*>(p.gate) + base;
  const TIO* x = static_cast<const TIO*>(p.x) + base;
  TIO* y = p.y ? static_cast<TIO*>(p.y) + base : nullptr;
  float h = p.ckpt[(b * p.blocks + k) * p.channels + c];
  for (int64_t t = t0; t < t1; ++t) {
    float a, w;
    gate_decay<LOG, sizeof(TIO) == 2>(to_f32(g[t * p.channels]), a, w);
    const float in = to_f32(x[t * p.channels]);
    if (p.hs) p.hs[base + t * p.channels] = h;
    h = fmaf(a, h, CONVEX ? w * in : in);
    if (y) y[t * p.channels] = from_f32<TIO>(h);
  }
}

template <typename TIO, bool LOG, bool CONVEX>
__global__ void gated_gradient_kernel(const GatedArgs p) {
  const int64_t c = (int64_t)(blockIdx.x % p.ctiles) * blockDim.x + threadIdx.x;
  const int64_t kb = blockIdx.x / p.ctiles, k = kb % p.blocks, b = kb / p.blocks;
  if (c >= p.channels) return;
  const int64_t t0 = k * kGatedBlock, t1 = min(p.len, t0 + kGatedBlock);
  const int64_t base = b * p.len * p.channels + c;
  float carry = p.enter[(b * p.blocks + k) * p.channels + c];
  for (int64_t t = t1 - 1; t >= t0; --t) {
    const int64_t at = base + t * p.channels;
    float a, w;
    gate_decay<LOG, sizeof(TIO) == 2>(to_f32(static_cast<const TIO*>(p.gate)[at]), a, w);
    const float x = to_f32(static_cast<const TIO*>(p.x)[at]);
    const float lam = to_f32(static_cast<const TIO*>(p.dy)[at]) + carry;
    const float before = CONVEX ? p.hs[at] - x : p.hs[at];
    static_cast<TIO*>(p.dx)[at] = from_f32<TIO>(CONVEX ? w * lam : lam);
    static_cast<TIO*>(p.dgate)[at] = from_f32<TIO>(lam * before * (LOG ? a : a * w));
    carry = a * lam;
  }
}

// One token per sequence, state in place.
template <typename TIO, bool LOG, bool CONVEX>
__global__ void gated_step_kernel(float* state, const TIO* x, const TIO* gate, TIO* y, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  float a, w;
  gate_decay<LOG, sizeof(TIO) == 2>(to_f32(gate[i]), a, w);
  const float in = to_f32(x[i]);
  const float h = fmaf(a, state[i], CONVEX ? w * in : in);
  state[i] = h;
  y[i] = from_f32<TIO>(h);
}

}  // namespace mamba
