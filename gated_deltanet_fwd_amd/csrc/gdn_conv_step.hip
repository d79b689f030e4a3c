// The conv1d + SiLU front-end's serving step on gfx950: gdn_conv_fwd's operation on sequences
// whose last W - 1 inputs are kept in a cache of windows between calls.
//
//   pre[c] = bias[c] + sum_{i<W} weight[c, i] x[t - (W-1) + i, c],  x before the call from the window
//   y[c]   = SiLU(pre[c]);  the window moves on by one row
//
// A lane owns 4 consecutive channels and runs a sequence's tokens in order, the window in registers.
// What bounds a batch is moving the windows and rows; a lane's taps (W floats a channel, more bytes
// than its bf16 rows) come from the L2, so in a batch with one token a sequence a lane takes two
// sequences and loads all of their rows at once: 256 sequences of 10,240 bf16 channels (42 MB) take 9.3
// us, 1.0 more with one a lane, 0.5 more with four; with 8 channels a lane 1.4 more, and a single sequence
// 3.9 us instead of 3.1. What bounds a run is the wait for each token's row, so the rows of STEP_U tokens
// are loaded together: 24 runs of up to 8 tokens 5.6 us, 1.2 more one by one. A run's rounds of four wait
// for each other: 700 tokens of 10,240 channels 215 us (29 MB), 5 such runs 237; 100 tokens 28.
#include "gdn_device.h"

namespace gdn {

constexpr int STEP_U = 4;

template <typename TI>
struct ConvRow { // a lane's channels as they are stored
  static constexpr int N = 4; // channels
  typedef TI vec __attribute__((ext_vector_type(N)));
};

// The lane's channels, taps and outputs.
template <typename TI, int W, bool SILU>
struct ConvLane {
  static constexpr int N = ConvRow<TI>::N, H = W - 1;
  typedef typename ConvRow<TI>::vec vec;
  const TI* x;
  TI *win, *y;
  int Cg;
  float wt[N][W], bs[N];
  __device__ __forceinline__ ConvLane(const ConvStepArgs& a, int c0) {
    int g = 0;
#pragma unroll
    for (int k = 1; k < 4; ++k) g += (k < a.n_groups && c0 >= a.goff[k]) ? 1 : 0;
    Cg = a.goff[g + 1] - a.goff[g];
    y = (TI*)a.y[g] + (c0 - a.goff[g]);
    x = (const TI*)a.x + c0;
    win = (TI*)a.win + c0;
    const f32x4* w = reinterpret_cast<const f32x4*>(a.w + (size_t)c0 * W); // N W floats
#pragma unroll
    for (int k = 0; k < N * W / 4; ++k) {
      const f32x4 r = w[k];
#pragma unroll
      for (int e = 0; e < 4; ++e) wt[(4 * k + e) / W][(4 * k + e) % W] = r[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) bs[e] = 0.f;
    if (a.b) {
      const f32x4* b = reinterpret_cast<const f32x4*>(a.b + c0);
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const f32x4 r = b[k];
#pragma unroll
        for (int e = 0; e < 4; ++e) bs[4 * k + e] = r[e];
      }
    }
  }
  // slot -1: zeros (slot 0 is read and masked, so that no branch stands between loads)
  __device__ __forceinline__ vec past(const ConvStepArgs& a, int slot, int j) const {
    const vec r = *reinterpret_cast<const vec*>(win + ((int64_t)max(slot, 0) * H + j) * a.C);
    typedef unsigned words __attribute__((ext_vector_type(sizeof(TI))));
    const unsigned m = slot < 0 ? 0u : ~0u;
    return __builtin_bit_cast(vec, __builtin_bit_cast(words, r) & m);
  }
  __device__ __forceinline__ vec row(const ConvStepArgs& a, int t) const {
    return *reinterpret_cast<const vec*>(x + (int64_t)t * a.xs);
  }
  __device__ __forceinline__ void store(const ConvStepArgs& a, int slot, const vec h[W]) const { // h[0 .. H - 1]
    if (slot < 0) return;
#pragma unroll
    for (int j = 0; j < H; ++j) *reinterpret_cast<vec*>(win + ((int64_t)slot * H + j) * a.C) = h[j];
  }
  __device__ __forceinline__ void out(int t, const vec h[W], bool bad) const {
    vec r;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float p = bs[e];
#pragma unroll
      for (int i = 0; i < W; ++i) p = __builtin_fmaf(wt[e][i], (float)h[i][e], p);
      // the hardware's reciprocal (about 1 ulp): p / inf is 0, as the sigmoid's end
      const float v = SILU ? p * __builtin_amdgcn_rcpf(1.f + __expf(-p)) : p;
      r[e] = (TI)(bad ? __builtin_nanf("") : v);
    }
    *reinterpret_cast<vec*>(y + (int64_t)t * Cg) = r;
  }
};

// One token a sequence, S sequences a lane (from blockIdx.y S on).
template <typename TI, int W, bool SILU, int S>
__global__ __launch_bounds__(256) void k_conv_step(ConvStepArgs a) {
  typedef ConvLane<TI, W, SILU> L;
  typedef typename L::vec vec;
  constexpr int H = W - 1;
  const int c0 = (blockIdx.x * 256 + threadIdx.x) * L::N;
  if (c0 >= a.C) return;
  for (int n0 = blockIdx.y * S; n0 < a.N; n0 += gridDim.y * S) {
    SeqSpan sp[S];
    vec h[S][W + 1];
    const L l(a, c0);
#pragma unroll
    for (int s = 0; s < S; ++s) sp[s] = seq_span(nullptr, a.slot_in, a.slot_out, min(n0 + s, a.N - 1), a.T, a.n_slots);
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < H; ++j) h[s][j] = l.past(a, sp[s].ok ? sp[s].in : 0, j);
      h[s][H] = l.row(a, sp[s].t0);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (n0 + s >= a.N) break;
      l.out(sp[s].t0, h[s], !sp[s].ok);
      l.store(a, sp[s].ok ? sp[s].out : -1, h[s] + 1);
    }
  }
}

// Runs of tokens.
template <typename TI, int W, bool SILU>
__global__ __launch_bounds__(256) void k_conv_run(ConvStepArgs a) {
  typedef ConvLane<TI, W, SILU> L;
  typedef typename L::vec vec;
  constexpr int H = W - 1, U = STEP_U;
  const int c0 = (blockIdx.x * 256 + threadIdx.x) * L::N;
  if (c0 >= a.C) return;
  const L l(a, c0);
  for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
    const SeqSpan sp = seq_span(a.cu, a.slot_in, a.slot_out, n, a.T, a.n_slots);
    vec h[U + W];
#pragma unroll
    for (int j = 0; j < U + W; ++j) h[j] = (vec)(TI)0.f;
    if (!sp.ok) {
      for (int t = sp.t0; t < sp.t1; ++t) l.out(t, h, true);
      continue;
    }
#pragma unroll
    for (int j = 0; j < H; ++j) h[j] = l.past(a, sp.in, j);
    for (int t = sp.t0; t < sp.t1; t += U) {
      int st[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tu = min(t + u, sp.t1 - 1);
        h[H + u] = l.row(a, tu);
        st[u] = a.slot_tok ? a.slot_tok[tu] : -1;
      }
      const int count = min(U, sp.t1 - t);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= count) break;
        const bool bad = st[u] < -1 || st[u] >= a.n_slots;
        l.out(t + u, h + u, bad);
        l.store(a, bad ? -1 : st[u], h + u + 1);
      }
      // the window after the block: rows count .. count + H - 1
      vec w[W];
#pragma unroll
      for (int j = 0; j < H; ++j) {
        w[j] = h[j + U];
#pragma unroll
        for (int u = 1; u < U; ++u)
          if (count == u) w[j] = h[j + u];
      }
#pragma unroll
      for (int j = 0; j < H; ++j) h[j] = w[j];
    }
    l.store(a, sp.out, h);
  }
}

template <typename TI, int W, bool SILU>
static int conv_step_w(const ConvStepArgs& a, hipStream_t s) {
  const int per = 256 * ConvRow<TI>::N, x = (a.C + per - 1) / per;
  const auto grid = [&](int n) { return dim3((unsigned)x, (unsigned)(n < 65535 ? n : 65535)); };
  // two sequences a lane where that leaves the CUs a few workgroups each
  if (a.cu || a.slot_tok) hipLaunchKernelGGL((k_conv_run<TI, W, SILU>), grid(a.N), dim3(256), 0, s, a);
  else if ((int64_t)x * a.N >= 4 * 256) hipLaunchKernelGGL((k_conv_step<TI, W, SILU, 2>), grid((a.N + 1) / 2), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_conv_step<TI, W, SILU, 1>), grid(a.N), dim3(256), 0, s, a);
  return (int)hipGetLastError();
}

template <typename TI>
static int conv_step_t(const ConvStepArgs& a, hipStream_t s) {
  switch (a.W * 2 + (a.silu ? 1 : 0)) {
    case 2: return conv_step_w<TI, 1, false>(a, s);
    case 3: return conv_step_w<TI, 1, true>(a, s);
    case 4: return conv_step_w<TI, 2, false>(a, s);
    case 5: return conv_step_w<TI, 2, true>(a, s);
    case 6: return conv_step_w<TI, 3, false>(a, s);
    case 7: return conv_step_w<TI, 3, true>(a, s);
    case 8: return conv_step_w<TI, 4, false>(a, s);
    default: return conv_step_w<TI, 4, true>(a, s);
  }
}

int launch_conv_step(const ConvStepArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == 0 ? conv_step_t<bf16>(a, s) : conv_step_t<float>(a, s);
}

} // namespace gdn
