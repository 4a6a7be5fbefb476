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
// The path is a stream: a token's channel costs 6 bytes (bf16) forward and 10
// backward, and about 20 and 40 instructions, so HBM bounds it as long as
// every element is read once and its gate computed once.  That shapes the
// kernels:
//   - A tile is 256 tokens by 64 bytes of channels (32 bf16, 16 fp32).  Its
//     tokens are 16 segments of 16, each walked by 16 lanes that hold 4 bytes
//     of channels.  A segment is the map h -> P h + H (P the product of its
//     gates, H its end state from zero); a and w x stay in registers between
//     the pass that forms the map and the pass that writes y.
//   - Tiles are staged in shared memory by cp.async, the next ones while this
//     one is worked on, by persistent CTAs, two per SM.
//   - One warp, a lane per channel, joins the segments' maps, publishes the
//     tile's map, looks back for the state that enters the tile, and hands
//     every segment its entering state.
// Time goes across CTAs: a tile's record in global memory is one 64-bit word
// per channel, (P, H), replaced by (0, state after the tile) once that is
// known; a map with P = 0 does not depend on what enters, so both are read the
// same way.  A word is written and read whole, so no fence or flag is needed:
// all bits set (which no (P, H) has) means not yet written.  The state that
// enters a tile is folded from the nearest record with P = 0 onwards, in time
// order: every tile rounds the same way whoever folds it, so results do not
// change from call to call.  Tiles are handed out by an atomic counter in time
// order, all chains (batch row, channel group) of a time before the next, so
// the smallest unfinished tile is always in a running CTA and the waits end.
// The backward pass walks the tiles in reverse with the adjoint's maps, from
// the states that enter every block of 256 tokens (checkpoints).
#pragma once

#include "common.cuh"

namespace mamba {

constexpr int kGatedBlock = MAMBA_GATED_SCAN_BLOCK;  // tokens of a tile
constexpr int kGatedThreads = 256;
constexpr int kGatedSegs = 16;                       // segments of a tile
constexpr int kGatedTok = kGatedBlock / kGatedSegs;  // tokens of a segment
constexpr int kGatedRow = 64;                        // bytes of a token's channels in a tile
// Two segments share a warp; 64 bytes between segments put them in different
// halves of the banks.
constexpr int kGatedSegBytes = kGatedTok * kGatedRow + 64;
constexpr int kGatedStream = kGatedSegs * kGatedSegBytes;  // bytes of one tensor's tile
constexpr int kGatedWindow = 8;                      // records looked at together
static_assert(kGatedThreads == kGatedSegs * 16, "16 lanes per segment");

struct GatedArgs {
  const void* x;
  const void* gate;
  const void* dy;
  const float* h0;       // [batch][channels] or NULL
  const float* dh;       // gradient of the final state, or NULL
  void* y;               // NULL: only checkpoints and final state
  float* final_state;    // or NULL
  float* ckpt;           // [batch][blocks][channels]: state entering each block, or NULL
  void* dx;
  void* dgate;
  float* dh0;
  unsigned long long* rec;  // [blocks][chains][channels of a tile] records, all bits set
  int* ticket;           // tiles handed out, starting at -1; NULL: one tile per chain, dealt by block index
  int64_t len, channels;
  int blocks;            // tiles along time
  int groups;            // channel groups
  int chains;            // batch * groups
  int jobs;              // chains * blocks
  uint64_t wait_limit_ns;
};

// ---------------------------------------------------------------------------
// gates
// ---------------------------------------------------------------------------
__device__ __forceinline__ float rcp_newton(float d) {
  // hardware reciprocal (1 ulp) and one Newton step: within 2^-24 of 1/d.  The
  // step is taken for bf16 data too: a state remembers thousands of gates, and
  // an error of one sign in each adds up in the float32 states.
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return fmaf(r, fmaf(-d, r, 1.0f), r);
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// a and 1 - a of a gate.  FAST (bf16 data): hardware exp2 (2^-22 of its value);
// else the CUDA library's functions.  Sigmoid: with e = exp(-g), a = 1/(1 + e)
// and 1 - a = e a, which has no cancellation; below g = -87, where e would
// overflow, a is zero.  Log form: near zero exp(g) - 1 by its series (next
// term below 2^-22 of it), which also keeps the bias of exp2 next to one out
// of long memories.
template <bool LOG, bool FAST>
__device__ __forceinline__ void gate_decay(float g, float& a, float& one_less) {
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (!LOG) {
    const float t = min_nan(FAST ? g * -kLog2e : -g, FAST ? 126.0f : 87.0f);
    const float e = FAST ? ex2_approx(t) : expf(t);
    const float r = rcp_newton(1.0f + e);
    one_less = e * r;
    a = t >= (FAST ? 126.0f : 87.0f) ? 0.0f : r;
  } else if constexpr (FAST) {
    const float big = ex2_approx(g * kLog2e);
    float p = fmaf(g, 1.0f / 720.0f, 1.0f / 120.0f);
    p = fmaf(p, g, 1.0f / 24.0f);
    p = fmaf(p, g, 1.0f / 6.0f);
    p = fmaf(p, g, 0.5f);
    p = fmaf(p, g, 1.0f);
    const bool small = fabsf(g) < 0.3f;
    a = small ? fmaf(g, p, 1.0f) : big;
    one_less = small ? -g * p : 1.0f - big;
  } else {
    a = expf(g);
    one_less = -expm1f(g);
  }
}

// 4 bytes of channels as floats
template <typename TIO>
struct Lane4 {
  static constexpr int kV = 4 / (int)sizeof(TIO);
  static __device__ __forceinline__ void get(uint32_t w, float (&v)[kV]) {
    if constexpr (kV == 1) {
      v[0] = __uint_as_float(w);
    } else {
      v[0] = __uint_as_float(w << 16);
      v[1] = __uint_as_float(w & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint32_t put(const float (&v)[kV]) {
    if constexpr (kV == 1) {
      return __float_as_uint(v[0]);
    } else {
      uint32_t w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(v[1]), "f"(v[0]));
      return w;
    }
  }
};

// ---------------------------------------------------------------------------
// tile loads and stores.  CB: bytes a copy moves, 16, 4, or 2 (plain loads),
// by the alignment of the tensors and of a row of channels.
// ---------------------------------------------------------------------------
template <int CB>
__device__ __forceinline__ void gated_copy(uint32_t dst, const unsigned char* src) {
  if constexpr (CB == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  } else if constexpr (CB == 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
  } else {
    const unsigned short v = *reinterpret_cast<const unsigned short*>(src);
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst), "h"(v) : "memory");
  }
}

// rows [0, n) x bytes [0, width) of a tile whose first byte is src
template <int CB>
__device__ __forceinline__ void gated_load(uint32_t dst, const unsigned char* src, int64_t pitch, int n, int width) {
  constexpr int kPer = kGatedRow / CB;                            // copies per row
  constexpr int kRows = kGatedThreads / kPer;                     // rows per round
  const int col = (threadIdx.x % kPer) * CB, r0 = threadIdx.x / kPer;
  if (col >= width) return;
  src += r0 * pitch + col;
#pragma unroll(CB == 16 ? 4 : 8)
  for (int i = 0; i < kGatedBlock / kRows; ++i) {
    const int r = r0 + i * kRows;
    if (r < n)
      gated_copy<CB>(dst + (r / kGatedTok) * kGatedSegBytes + (r % kGatedTok) * kGatedRow + col, src);
    src += kRows * pitch;
  }
}

// one lane's 4 bytes (or the part of them inside the row)
template <int CB>
__device__ __forceinline__ void gated_store(unsigned char* dst, uint32_t w, int left) {
  if constexpr (CB >= 4) {
    *reinterpret_cast<uint32_t*>(dst) = w;
  } else {
    reinterpret_cast<unsigned short*>(dst)[0] = (unsigned short)w;
    if (left > 2) reinterpret_cast<unsigned short*>(dst)[1] = (unsigned short)(w >> 16);
  }
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// ---------------------------------------------------------------------------
// records
// ---------------------------------------------------------------------------
__device__ __forceinline__ void rec_put(unsigned long long* p, float P, float H) {
  const uint32_t pb = P == P ? __float_as_uint(P) : 0x7fffffffu;  // a NaN is not "not yet written"
  const unsigned long long v = ((unsigned long long)pb << 32) | __float_as_uint(H);
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long rec_get(const unsigned long long* p) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}

// The state that enters the tile of `own`: from the nearest of the `before`
// tiles before it whose record has P = 0, through the maps in between.
// Records lie `stride` apart.  Called by a whole warp, a lane per channel.
__device__ __forceinline__ float gated_look_back(const unsigned long long* own, int before, int64_t stride,
                                                 bool active, uint64_t limit_ns) {
  float h = 0.0f;
  bool done = !active;
  uint64_t t0 = 0;
  for (uint32_t round = 0;; ++round) {
    if (!done) {
      unsigned long long r[kGatedWindow];
#pragma unroll
      for (int i = 0; i < kGatedWindow; ++i) r[i] = i < before ? rec_get(own - (i + 1) * stride) : 0ull;
      int found = -1;
      bool ready = true;
#pragma unroll
      for (int i = 0; i < kGatedWindow; ++i) {
        const uint32_t pb = (uint32_t)(r[i] >> 32);
        ready = ready && pb != 0xffffffffu && i < before;
        if (ready && found < 0 && __uint_as_float(pb) == 0.0f) found = i;
      }
      if (found >= 0) {
        done = true;
#pragma unroll
        for (int i = kGatedWindow - 1; i >= 0; --i)
          if (i <= found) h = fmaf(__uint_as_float((uint32_t)(r[i] >> 32)), h, __uint_as_float((uint32_t)r[i]));
      }
    }
    if (__all_sync(0xffffffffu, done)) return h;
    if ((round & 63u) == 63u) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > limit_ns) {
        record_device_error(MAMBA_ERR_TIMEOUT);
        return h;
      }
    }
  }
}

// Tile `job` of a launch: chain (batch row, channel group) and time block.
struct GatedTile {
  int64_t at;   // element index of its first token's first channel
  int k, chain; // block counted in walking order, chain
  int c0;       // first channel
  int b;
  int n;        // tokens
};
template <typename TIO, bool REVERSE>
__device__ __forceinline__ GatedTile gated_tile(const GatedArgs& p, int job) {
  GatedTile t;
  t.k = job / p.chains;
  t.chain = job - t.k * p.chains;
  t.b = t.chain / p.groups;
  t.c0 = (t.chain - t.b * p.groups) * (kGatedRow / (int)sizeof(TIO));
  const int block = REVERSE ? p.blocks - 1 - t.k : t.k;
  const int64_t t0 = (int64_t)block * kGatedBlock;
  t.n = (int)min((int64_t)kGatedBlock, p.len - t0);
  t.at = ((int64_t)t.b * p.len + t0) * p.channels + t.c0;
  return t;
}

// Shared memory: the stages, then the segments' maps and entering states.
template <typename TIO>
struct GatedSmem {
  static constexpr int kChan = kGatedRow / (int)sizeof(TIO);
  static constexpr int kSmall = kGatedSegs * kChan * 4;  // one float per segment and channel
  static constexpr int fwd(int stages) { return stages * 2 * kGatedStream + 3 * kSmall + 64; }
  static constexpr int bwd(int stages) { return stages * 3 * kGatedStream + 5 * kSmall + 64; }
};
constexpr int kGatedFwdStages = 2;
constexpr int kGatedBwdStages = 2;

// Tiles of a CTA: S to start with, then one for each that is done.  With one
// tile per CTA at most, each takes just one, so that none waits behind another.
// One tile per chain: no order is needed, and tiles are dealt by block index.
template <int S>
__device__ __forceinline__ void gated_first(const GatedArgs& p, int* queue) {
  if (threadIdx.x != 0) return;
  const bool ahead = p.jobs > (int)gridDim.x;
  int first = blockIdx.x, step = gridDim.x;
  if (p.ticket) {
    first = atomicAdd(p.ticket, ahead ? S : 1) + 1;
    step = ahead ? 1 : p.jobs;
  }
  queue[0] = first;
#pragma unroll
  for (int s = 1; s < S; ++s) queue[s] = min(first + s * step, p.jobs);
}
template <int S>
__device__ __forceinline__ int gated_next(const GatedArgs& p, int job) {
  if (p.jobs <= (int)gridDim.x) return p.jobs;
  return p.ticket ? atomicAdd(p.ticket, 1) + 1 : min(job + S * (int)gridDim.x, p.jobs);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename TIO, bool LOG, bool CONVEX, int CB>
__global__ void __launch_bounds__(kGatedThreads, 2) gated_scan_kernel(const GatedArgs p) {
  using L4 = Lane4<TIO>;
  constexpr int V = L4::kV, kChan = GatedSmem<TIO>::kChan, kES = (int)sizeof(TIO), S = kGatedFwdStages;
  extern __shared__ __align__(16) unsigned char smem[];
  float* seg_p = reinterpret_cast<float*>(smem + S * 2 * kGatedStream);  // [segment][channel]
  float* seg_h = seg_p + kGatedSegs * kChan;
  float* seg_in = seg_h + kGatedSegs * kChan;
  int* queue = reinterpret_cast<int*>(seg_in + kGatedSegs * kChan);
  const int tid = threadIdx.x, seg = tid >> 4, sl = tid & 15;
  const uint32_t stage0 = smem_addr(smem);
  const uint32_t mine = seg * kGatedSegBytes + sl * 4;
  const int64_t pitch = p.channels * kES;
  griddep_launch_dependents();
  griddep_wait();

  // several tiles per CTA: one is worked on while the next is loaded
  gated_first<S>(p, queue);
  __syncthreads();
  auto load = [&](int stage) {
    const int job = queue[stage];
    if (job < p.jobs) {
      const GatedTile t = gated_tile<TIO, false>(p, job);
      const int width = (int)min((int64_t)kGatedRow, (p.channels - t.c0) * kES);
      const uint32_t to = stage0 + stage * 2 * kGatedStream;
      gated_load<CB>(to, static_cast<const unsigned char*>(p.gate) + t.at * kES, pitch, t.n, width);
      gated_load<CB>(to + kGatedStream, static_cast<const unsigned char*>(p.x) + t.at * kES, pitch, t.n, width);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < S; ++s) load(s);

  for (int stage = 0;; stage = stage + 1 == S ? 0 : stage + 1) {
    const int job = queue[stage];
    if (job >= p.jobs) break;
    const GatedTile t = gated_tile<TIO, false>(p, job);
    cp_async_wait<S - 1>();
    __syncthreads();
    int next = 0;
    if (tid == 32) next = gated_next<S>(p, job);

    // the segment's gates and inputs, and its map
    const uint32_t from = stage0 + stage * 2 * kGatedStream + mine;
    const int n = min(kGatedTok, t.n - seg * kGatedTok);
    float a[kGatedTok][V], b[kGatedTok][V], P[V], H[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.0f, H[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < kGatedTok; ++i) {
      float g[V], x[V], w;
      L4::get(lds32(from + i * kGatedRow), g);
      L4::get(lds32(from + kGatedStream + i * kGatedRow), x);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gate_decay<LOG, sizeof(TIO) == 2>(g[v], a[i][v], w);
        b[i][v] = CONVEX ? w * x[v] : x[v];
        if (i < n) {
          H[v] = fmaf(a[i][v], H[v], b[i][v]);
          P[v] *= a[i][v];
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      seg_p[seg * kChan + sl * V + v] = P[v];
      seg_h[seg * kChan + sl * V + v] = H[v];
    }
    if (tid == 32) queue[stage] = next;
    __syncthreads();
    load(stage);

    if (tid < 32) {
      const bool active = tid < kChan && t.c0 + tid < p.channels;
      const int ch = tid < kChan ? tid : 0;
      unsigned long long* rec = p.rec + ((int64_t)t.k * p.chains + t.chain) * kChan + ch;
      const int64_t state_at = (int64_t)t.b * p.channels + t.c0 + ch;
      float h = 0.0f;
      if (t.k == 0) {
        if (active && p.h0) h = p.h0[state_at];
      } else {
        float tp = 1.0f, th = 0.0f;
#pragma unroll
        for (int s = 0; s < kGatedSegs; ++s) {
          th = fmaf(seg_p[s * kChan + ch], th, seg_h[s * kChan + ch]);
          tp *= seg_p[s * kChan + ch];
        }
        if (active && t.k + 1 < p.blocks) rec_put(rec, tp, th);
        h = gated_look_back(rec, t.k, (int64_t)p.chains * kChan, active, p.wait_limit_ns);
      }
      if (active && p.ckpt) p.ckpt[((int64_t)t.b * p.blocks + t.k) * p.channels + t.c0 + ch] = h;
      // the next tile's entering state, rounded as a reader of (P, H) rounds it
      float tp = 1.0f, th = 0.0f;
      const float h_in = h;
#pragma unroll
      for (int s = 0; s < kGatedSegs; ++s) {
        const float sp = seg_p[s * kChan + ch], sh = seg_h[s * kChan + ch];
        if (tid < kChan) seg_in[s * kChan + ch] = h;
        h = fmaf(sp, h, sh);
        th = fmaf(sp, th, sh);
        tp *= sp;
      }
      const float after = fmaf(tp, h_in, th);
      if (active) {
        if (t.k + 1 < p.blocks) rec_put(rec, 0.0f, after);
        else if (p.final_state) p.final_state[state_at] = after;
      }
    }
    __syncthreads();

    if (p.y && t.c0 + sl * V < p.channels) {
      float h[V];
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = seg_in[seg * kChan + sl * V + v];
      unsigned char* y = static_cast<unsigned char*>(p.y) + (t.at + (int64_t)seg * kGatedTok * p.channels + sl * V) * kES;
      const int left = (int)min((int64_t)4, (p.channels - t.c0 - sl * V) * kES);
#pragma unroll
      for (int i = 0; i < kGatedTok; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], h[v], b[i][v]);
        if (i < n) gated_store<CB>(y, L4::put(h), left);
        y += pitch;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// The adjoint's map of a segment takes c = a_{t+1} lam_{t+1} of the token after
// it to a_s lam_s of its first token s: c -> P c + R, R = sum of dy_t a_s..a_t.
template <typename TIO, bool LOG, bool CONVEX, int CB>
__global__ void __launch_bounds__(kGatedThreads, 2) gated_backward_kernel(const GatedArgs p) {
  using L4 = Lane4<TIO>;
  constexpr int V = L4::kV, kChan = GatedSmem<TIO>::kChan, kES = (int)sizeof(TIO), S = kGatedBwdStages;
  constexpr bool kFast = sizeof(TIO) == 2;
  extern __shared__ __align__(16) unsigned char smem[];
  float* seg_p = reinterpret_cast<float*>(smem + S * 3 * kGatedStream);  // [segment][channel]
  float* seg_h = seg_p + kGatedSegs * kChan;
  float* seg_r = seg_h + kGatedSegs * kChan;
  float* seg_in = seg_r + kGatedSegs * kChan;   // state entering from the left
  float* seg_adj = seg_in + kGatedSegs * kChan; // adjoint entering from the right
  int* queue = reinterpret_cast<int*>(seg_adj + kGatedSegs * kChan);
  const int tid = threadIdx.x, seg = tid >> 4, sl = tid & 15;
  const uint32_t stage0 = smem_addr(smem);
  const uint32_t mine = seg * kGatedSegBytes + sl * 4;
  const int64_t pitch = p.channels * kES;
  griddep_launch_dependents();
  griddep_wait();

  gated_first<S>(p, queue);
  __syncthreads();
  auto load = [&](int stage) {
    const int job = queue[stage];
    if (job < p.jobs) {
      const GatedTile t = gated_tile<TIO, true>(p, job);
      const int width = (int)min((int64_t)kGatedRow, (p.channels - t.c0) * kES);
      const uint32_t to = stage0 + stage * 3 * kGatedStream;
      gated_load<CB>(to, static_cast<const unsigned char*>(p.gate) + t.at * kES, pitch, t.n, width);
      gated_load<CB>(to + kGatedStream, static_cast<const unsigned char*>(p.x) + t.at * kES, pitch, t.n, width);
      gated_load<CB>(to + 2 * kGatedStream, static_cast<const unsigned char*>(p.dy) + t.at * kES, pitch, t.n, width);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < S; ++s) load(s);

  for (int stage = 0;; stage = stage + 1 == S ? 0 : stage + 1) {
    const int job = queue[stage];
    if (job >= p.jobs) break;
    const GatedTile t = gated_tile<TIO, true>(p, job);
    cp_async_wait<S - 1>();
    __syncthreads();
    int next = 0;
    if (tid == 32) next = gated_next<S>(p, job);

    const uint32_t from = stage0 + stage * 3 * kGatedStream + mine;
    const int n = min(kGatedTok, t.n - seg * kGatedTok);
    float a[kGatedTok][V], b[kGatedTok][V], P[V], H[V], R[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.0f, H[v] = 0.0f, R[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < kGatedTok; ++i) {
      float g[V], x[V], dy[V], w;
      L4::get(lds32(from + i * kGatedRow), g);
      L4::get(lds32(from + kGatedStream + i * kGatedRow), x);
      L4::get(lds32(from + 2 * kGatedStream + i * kGatedRow), dy);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gate_decay<LOG, kFast>(g[v], a[i][v], w);
        b[i][v] = CONVEX ? w * x[v] : x[v];
        if (i < n) {
          H[v] = fmaf(a[i][v], H[v], b[i][v]);
          P[v] *= a[i][v];
          R[v] = fmaf(dy[v], P[v], R[v]);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      seg_p[seg * kChan + sl * V + v] = P[v];
      seg_h[seg * kChan + sl * V + v] = H[v];
      seg_r[seg * kChan + sl * V + v] = R[v];
    }
    __syncthreads();

    const int lane = tid & 31;
    const bool active = lane < kChan && t.c0 + lane < p.channels;
    const int ch = lane < kChan ? lane : 0;
    const int64_t state_at = (int64_t)t.b * p.channels + t.c0 + ch;
    if (tid < 32) {  // the adjoint, from the right
      unsigned long long* rec = p.rec + ((int64_t)t.k * p.chains + t.chain) * kChan + ch;
      float c = 0.0f;
      if (t.k == 0) {
        if (active && p.dh) c = p.dh[state_at];
      } else {
        float tp = 1.0f, tr = 0.0f;
#pragma unroll
        for (int s = kGatedSegs - 1; s >= 0; --s) {
          tr = fmaf(seg_p[s * kChan + ch], tr, seg_r[s * kChan + ch]);
          tp *= seg_p[s * kChan + ch];
        }
        if (active && t.k + 1 < p.blocks) rec_put(rec, tp, tr);
        c = gated_look_back(rec, t.k, (int64_t)p.chains * kChan, active, p.wait_limit_ns);
      }
      float tp = 1.0f, tr = 0.0f;
      const float c_in = c;
#pragma unroll
      for (int s = kGatedSegs - 1; s >= 0; --s) {
        const float sp = seg_p[s * kChan + ch], sr = seg_r[s * kChan + ch];
        if (lane < kChan) seg_adj[s * kChan + ch] = c;
        c = fmaf(sp, c, sr);
        tr = fmaf(sp, tr, sr);
        tp *= sp;
      }
      const float after = fmaf(tp, c_in, tr);
      if (active) {
        if (t.k + 1 < p.blocks) rec_put(rec, 0.0f, after);
        else if (p.dh0) p.dh0[state_at] = after;
      }
    } else if (tid < 64) {  // the states, from the checkpoint
      const int block = p.blocks - 1 - t.k;
      float h = active ? p.ckpt[((int64_t)t.b * p.blocks + block) * p.channels + t.c0 + ch] : 0.0f;
#pragma unroll
      for (int s = 0; s < kGatedSegs; ++s) {
        if (lane < kChan) seg_in[s * kChan + ch] = h;
        h = fmaf(seg_p[s * kChan + ch], h, seg_h[s * kChan + ch]);
      }
    }
    __syncthreads();

    if (t.c0 + sl * V < p.channels) {
      // b becomes h_{t-1} (minus x_t when convex)
      float h[V], c[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = seg_in[seg * kChan + sl * V + v];
        c[v] = seg_adj[seg * kChan + sl * V + v];
      }
#pragma unroll
      for (int i = 0; i < kGatedTok; ++i) {
        float x[V];
        if (CONVEX) L4::get(lds32(from + kGatedStream + i * kGatedRow), x);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float before = h[v];
          h[v] = fmaf(a[i][v], h[v], b[i][v]);
          b[i][v] = CONVEX ? before - x[v] : before;
        }
      }
      const int64_t at = (t.at + (int64_t)seg * kGatedTok * p.channels + sl * V) * kES;
      unsigned char* dx = static_cast<unsigned char*>(p.dx) + at + (kGatedTok - 1) * pitch;
      unsigned char* dg = static_cast<unsigned char*>(p.dgate) + at + (kGatedTok - 1) * pitch;
      const int left = (int)min((int64_t)4, (p.channels - t.c0 - sl * V) * kES);
#pragma unroll
      for (int i = kGatedTok - 1; i >= 0; --i) {
        if (i < n) {
          float g[V], dy[V], ox[V], og[V];
          if (CONVEX || !LOG) L4::get(lds32(from + i * kGatedRow), g);
          L4::get(lds32(from + 2 * kGatedStream + i * kGatedRow), dy);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            float again, w = 1.0f;
            if (CONVEX || !LOG) gate_decay<LOG, kFast>(g[v], again, w);
            const float lam = dy[v] + c[v];
            c[v] = a[i][v] * lam;
            ox[v] = CONVEX ? w * lam : lam;
            og[v] = (LOG ? c[v] : c[v] * w) * b[i][v];
          }
          gated_store<CB>(dx, L4::put(ox), left);
          gated_store<CB>(dg, L4::put(og), left);
        }
        dx -= pitch;
        dg -= pitch;
      }
    }
    if (tid == 32) queue[stage] = next;
    __syncthreads();  // the stage is read to the end
    load(stage);
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
