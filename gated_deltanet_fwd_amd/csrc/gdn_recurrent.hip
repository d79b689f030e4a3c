// The gated delta rule, recurrent, on cached FP32 states (gfx950): one token a sequence when
// decoding, short runs when drafted tokens are checked or a prompt is extended. Per token and
// value head, with a = exp(g), raw rows k and q and their inverse norms rk, rq (1 without the norm):
//
//   s1 = rk S^T k,  s2 = rq S^T q            (one pass over the old state)
//   u  = beta (v - a s1)
//   o  = a s2 + rq rk (q.k) u                (= S_new^T q rq)
//   S  = a S + k (rk u)^T
//
// Columns of S (value indices) never mix, so a wave owns NC columns of one head's state and keeps
// them in registers from the first token to the last: lane (kg, cg) holds 4 consecutive columns of
// D / KG rows, a state row's NC columns lie in consecutive lanes. Sums over the rows (keys) run
// inside the lane, then over the key groups across lanes.
#include "gdn_device.h"

namespace gdn {

// Sum over the lanes that agree in the low bits below LR (all key groups), in every lane.
template <int LR>
__device__ __forceinline__ float key_sum(float x) {
  if constexpr (LR <= 2) x += __shfl_xor(x, 2);
  if constexpr (LR <= 4) x += __shfl_xor(x, 4);
  x += __shfl_xor(x, 8);
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

template <typename TI, int N>
__device__ __forceinline__ void load_keys(const TI* p, float v[N]) {
  typedef TI vec __attribute__((ext_vector_type(N)));
  const vec r = *reinterpret_cast<const vec*>(p);
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = (float)r[e];
}

template <typename TI, int D, int NC>
__global__ __launch_bounds__(256) void k_recurrent(RecurrentArgs a) {
  constexpr int LR = NC / 4;  // lanes along a state row
  constexpr int KG = 64 / LR; // key groups
  constexpr int KPL = D / KG; // keys per lane
  constexpr int CB = D / NC;  // waves per state
  const int lane = threadIdx.x & 63;
  const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t sh = wid / CB; // (sequence, head)
  if (sh >= (int64_t)a.N * a.HV) return;
  const int n = (int)(sh / a.HV), h = (int)(sh - (int64_t)n * a.HV);
  const int j = h / a.G;
  const int key0 = (lane / LR) * KPL;
  const int col0 = (int)(wid - sh * CB) * NC + (lane % LR) * 4;
  TI* o = (TI*)a.o + (int64_t)h * D + col0;
  const int64_t os = (int64_t)a.HV * D;
  const SeqSpan sp = seq_span(a.cu, a.slot_in, a.slot_out, n, a.T, a.n_slots);
  const float nan = __builtin_nanf("");
  if (!sp.ok) {
    const float v[4] = {nan, nan, nan, nan};
    if (key0 == 0)
      for (int64_t t = sp.t0; t < sp.t1; ++t) IO<TI>::store4(o + t * os, v);
    return;
  }
  const int64_t hd = (int64_t)a.HV * D * D, at = (int64_t)h * D * D + (int64_t)key0 * D + col0;
  float S[KPL][4];
  if (sp.in >= 0) {
    const float* p = a.states + sp.in * hd + at;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const f32x4 r = *reinterpret_cast<const f32x4*>(p + i * D);
#pragma unroll
      for (int c = 0; c < 4; ++c) S[i][c] = r[c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < KPL; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[i][c] = 0.f;
  }
  const TI* q = (const TI*)a.q + (int64_t)j * D + key0;
  const TI* k = (const TI*)a.k + (int64_t)j * D + key0;
  const TI* v = (const TI*)a.v + (int64_t)h * D + col0;
  for (int64_t t = sp.t0; t < sp.t1; ++t) {
    float kt[KPL], qt[KPL], vt[4];
    load_keys<TI, KPL>(k + t * a.ks, kt);
    load_keys<TI, KPL>(q + t * a.qs, qt);
    load_keys<TI, 4>(v + t * a.vs, vt);
    const float al = __expf(a.g[t * a.HV + h]), be = a.beta[t * a.HV + h];
    const int st = a.slot_tok ? a.slot_tok[t] : -1;
    float kk = 0.f, qq = 0.f, qk = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      kk = __builtin_fmaf(kt[i], kt[i], kk);
      qq = __builtin_fmaf(qt[i], qt[i], qq);
      qk = __builtin_fmaf(qt[i], kt[i], qk);
    }
    float rk = 1.f, rq = 1.f;
    if (a.l2norm) {
      rk = 1.f / sqrtf(key_sum<LR>(kk) + 1e-6f);
      rq = 1.f / sqrtf(key_sum<LR>(qq) + 1e-6f);
    }
    qk = key_sum<LR>(qk) * rq * rk;
    float s1[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KPL; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s1[c] = __builtin_fmaf(S[i][c], kt[i], s1[c]);
        s2[c] = __builtin_fmaf(S[i][c], qt[i], s2[c]);
      }
    float u[4], out[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      s1[c] = key_sum<LR>(s1[c]) * rk;
      s2[c] = key_sum<LR>(s2[c]) * rq;
      u[c] = be * (vt[c] - al * s1[c]);
      out[c] = __builtin_fmaf(al, s2[c], qk * u[c]);
      u[c] *= rk;
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[i][c] = __builtin_fmaf(kt[i], u[c], al * S[i][c]);
    const bool bad = st < -1 || st >= a.n_slots;
    if (bad) out[0] = out[1] = out[2] = out[3] = nan;
    if (key0 == 0) IO<TI>::store4(o + t * os, out);
    if (st >= 0 && !bad) {
      float* p = a.states + st * hd + at;
#pragma unroll
      for (int i = 0; i < KPL; ++i) *reinterpret_cast<f32x4*>(p + i * D) = f32x4{S[i][0], S[i][1], S[i][2], S[i][3]};
    }
  }
  if (sp.out >= 0) {
    float* p = a.states + sp.out * hd + at;
#pragma unroll
    for (int i = 0; i < KPL; ++i) *reinterpret_cast<f32x4*>(p + i * D) = f32x4{S[i][0], S[i][1], S[i][2], S[i][3]};
  }
}

template <typename TI, int D>
static int recurrent_t(const RecurrentArgs& a, hipStream_t s) {
  constexpr int NC = 32;
  const int64_t waves = (int64_t)a.N * a.HV * (D / NC);
  hipLaunchKernelGGL((k_recurrent<TI, D, NC>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, a);
  return (int)hipGetLastError();
}

int launch_recurrent(const RecurrentArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == 0) return a.D == 128 ? recurrent_t<bf16, 128>(a, s) : recurrent_t<bf16, 64>(a, s);
  return a.D == 128 ? recurrent_t<float, 128>(a, s) : recurrent_t<float, 64>(a, s);
}

} // namespace gdn
