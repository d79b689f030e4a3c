// The conv1d + SiLU front-end's serving step on gfx950: gdn_conv_fwd's operation on sequences
// whose last W - 1 inputs are kept in a cache of windows between calls.
//
//   pre[c] = bias[c] + sum_{i<W} weight[c, i] x[t - (W-1) + i, c],  x before the call from the window
//   y[c]   = SiLU(pre[c]);  the window moves on by one row
//
// A lane owns 4 consecutive channels of one sequence and runs its tokens in order, the window in
// registers.
#include "gdn_device.h"

namespace gdn {

constexpr int CS_CPL = 4; // channels per lane

template <typename TI>
struct Row4 { // 4 consecutive values of a row as they are stored (8 or 16 bytes)
  typedef TI vec __attribute__((ext_vector_type(4)));
};

template <typename TI, int W, bool SILU>
__global__ __launch_bounds__(256) void k_conv_step(ConvStepArgs a) {
  typedef typename Row4<TI>::vec vec;
  constexpr int H = W - 1;
  const int c0 = (blockIdx.x * 256 + threadIdx.x) * CS_CPL;
  if (c0 >= a.C) return;
  int g = 0;
#pragma unroll
  for (int k = 1; k < 4; ++k) g += (k < a.n_groups && c0 >= a.goff[k]) ? 1 : 0;
  const int Cg = a.goff[g + 1] - a.goff[g];
  TI* y = (TI*)a.y[g] + (c0 - a.goff[g]);
  const TI* x = (const TI*)a.x + c0;
  TI* win = (TI*)a.win + c0;
  float wt[CS_CPL][W], bs[CS_CPL];
#pragma unroll
  for (int e = 0; e < CS_CPL; ++e) {
#pragma unroll
    for (int i = 0; i < W; ++i) wt[e][i] = a.w[(size_t)(c0 + e) * W + i];
    bs[e] = a.b ? a.b[c0 + e] : 0.f;
  }
  for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
    const SeqSpan sp = seq_span(a.cu, a.slot_in, a.slot_out, n, a.T, a.n_slots);
    if (!sp.ok) {
      const vec nan4 = (vec)(TI)__builtin_nanf("");
      for (int t = sp.t0; t < sp.t1; ++t) *reinterpret_cast<vec*>(y + (int64_t)t * Cg) = nan4;
      continue;
    }
    vec h[W]; // the window's rows, the newest last; h[H] is the current token
    if constexpr (H > 0) {
#pragma unroll
      for (int j = 0; j < H; ++j)
        h[j] = sp.in < 0 ? (vec)(TI)0.f
                         : *reinterpret_cast<const vec*>(win + ((int64_t)sp.in * H + j) * a.C);
    }
    for (int t = sp.t0; t < sp.t1; ++t) {
      h[H] = *reinterpret_cast<const vec*>(x + t * a.xs);
      const int st = a.slot_tok ? a.slot_tok[t] : -1;
      vec out;
#pragma unroll
      for (int e = 0; e < CS_CPL; ++e) {
        float p = bs[e];
#pragma unroll
        for (int i = 0; i < W; ++i) p = __builtin_fmaf(wt[e][i], (float)h[i][e], p);
        const float r = SILU ? p / (1.f + __expf(-p)) : p;
        out[e] = (TI)(st < -1 || st >= a.n_slots ? __builtin_nanf("") : r);
      }
      *reinterpret_cast<vec*>(y + (int64_t)t * Cg) = out;
#pragma unroll
      for (int j = 0; j < H; ++j) h[j] = h[j + 1];
      if constexpr (H > 0) {
        if (st >= 0 && st < a.n_slots) {
#pragma unroll
          for (int j = 0; j < H; ++j) *reinterpret_cast<vec*>(win + ((int64_t)st * H + j) * a.C) = h[j];
        }
      }
    }
    if constexpr (H > 0) {
      if (sp.out >= 0) {
#pragma unroll
        for (int j = 0; j < H; ++j) *reinterpret_cast<vec*>(win + ((int64_t)sp.out * H + j) * a.C) = h[j];
      }
    }
  }
}

template <typename TI>
static int conv_step_t(const ConvStepArgs& a, hipStream_t s) {
  const dim3 grid((a.C + 256 * CS_CPL - 1) / (256 * CS_CPL), a.N < 65535 ? a.N : 65535), blk(256);
  switch (a.W * 2 + (a.silu ? 1 : 0)) {
    case 2: hipLaunchKernelGGL((k_conv_step<TI, 1, false>), grid, blk, 0, s, a); break;
    case 3: hipLaunchKernelGGL((k_conv_step<TI, 1, true>), grid, blk, 0, s, a); break;
    case 4: hipLaunchKernelGGL((k_conv_step<TI, 2, false>), grid, blk, 0, s, a); break;
    case 5: hipLaunchKernelGGL((k_conv_step<TI, 2, true>), grid, blk, 0, s, a); break;
    case 6: hipLaunchKernelGGL((k_conv_step<TI, 3, false>), grid, blk, 0, s, a); break;
    case 7: hipLaunchKernelGGL((k_conv_step<TI, 3, true>), grid, blk, 0, s, a); break;
    case 8: hipLaunchKernelGGL((k_conv_step<TI, 4, false>), grid, blk, 0, s, a); break;
    default: hipLaunchKernelGGL((k_conv_step<TI, 4, true>), grid, blk, 0, s, a); break;
  }
  return (int)hipGetLastError();
}

int launch_conv_step(const ConvStepArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == 0 ? conv_step_t<bf16>(a, s) : conv_step_t<float>(a, s);
}

} // namespace gdn
