// Norms of the q and k heads with the position rotation, forward and backward (gfx950). Per head
// row x of a token at position p, c = 1/D (RMS) or 1 (L2), r = 1/sqrt(c sum x^2 + eps):
//
//   n = x r,  z = n w,  y = m R(p f) z           (R turns the pairs of the first RD values)
//   dz = m R(-p f) dy,  dn = dz w,  dw = sum dz n,  dx = r (dn - c n (n.dn))
//
// A row is held by a group of 8, 16 or 32 lanes, 8 values a lane. With pairs half the rotary dim
// apart a lane takes 4 consecutive values of each half, so that both values of a pair and the 4
// frequencies it needs are in the lane in both layouts. A group takes one token and `hc` of its
// q/k heads, so the token's cosines and sines are computed once for all of them.
//
// The angle is exact: a frequency is a 64-bit fraction of a turn per position, and the product with
// the position modulo 2^64 drops whole turns. Its top 32 bits give the quadrant and a remainder of
// at most 1/8 turn, where the Taylor polynomials of sine and cosine to x^9 and x^10 are off by less
// than 2e-9 and 2e-10.
#include "gdn_device.h"

namespace gdn {

template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
  const auto dpp = [](float v, auto ctrl) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  x += dpp(x, std::integral_constant<int, 0xB1>{});  // lane ^ 1
  x += dpp(x, std::integral_constant<int, 0x4E>{});  // lane ^ 2
  x += dpp(x, std::integral_constant<int, 0x141>{}); // 7 - lane within 8: the other quad
  if constexpr (LPR >= 16) x += dpp(x, std::integral_constant<int, 0x140>{}); // 15 - lane within 16
  if constexpr (LPR >= 32) x += __shfl_xor(x, 16);
  return x;
}

// cos and sin of the angle pos * freq (freq in 2^-64 turns).
__device__ __forceinline__ void turn_cs(int pos, uint64_t freq, float& c, float& s) {
  const uint32_t top = (uint32_t)(((uint64_t)(int64_t)pos * freq) >> 32) + 0x20000000u; // shifted by 1/8 turn
  const uint32_t quad = top >> 30;
  const float x = (float)((int)(top & 0x3fffffffu) - 0x20000000) * 1.46291807926715968105e-09f; // 2 pi / 2^32
  const float x2 = x * x;
  float sp = __builtin_fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);
  sp = __builtin_fmaf(x2, sp, 8.33333333e-3f);
  sp = __builtin_fmaf(x2, sp, -1.66666667e-1f);
  sp = __builtin_fmaf(x2 * x, sp, x);
  float cp = __builtin_fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);
  cp = __builtin_fmaf(x2, cp, -1.38888889e-3f);
  cp = __builtin_fmaf(x2, cp, 4.16666667e-2f);
  cp = __builtin_fmaf(x2, cp, -0.5f);
  cp = __builtin_fmaf(x2, cp, 1.f);
  const float cc = quad & 1 ? sp : cp, ss = quad & 1 ? cp : sp;
  c = (quad + 1) & 2 ? -cc : cc; // quadrants 1 and 2
  s = quad & 2 ? -ss : ss;       // quadrants 2 and 3
}

// Where a lane's 8 values lie in a row: values 0..3 at o1, 4..7 at o2.
struct RowMap {
  int o1, o2;
  bool on, rot;
};
template <bool HALF>
__device__ __forceinline__ RowMap row_map(int j, int D, int RD) {
  RowMap m;
  m.on = 8 * j < D;
  m.rot = 8 * j < RD;
  m.o1 = HALF && m.rot ? 4 * j : 8 * j;
  m.o2 = HALF && m.rot ? RD / 2 + 4 * j : 8 * j + 4;
  return m;
}

template <typename TI>
__device__ __forceinline__ void load4f(const TI* p, float* v) {
  typedef TI vec __attribute__((ext_vector_type(4)));
  const vec r = *reinterpret_cast<const vec*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)r[e];
}

template <typename TI, bool HALF>
__device__ __forceinline__ void load_row(const TI* p, const RowMap& m, float v[8]) {
  if (!m.on) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  } else if constexpr (HALF) {
    load4f(p + m.o1, v);
    load4f(p + m.o2, v + 4);
  } else {
    IO<TI>::load8f(p + m.o1, v);
  }
}

template <typename TI, bool HALF>
__device__ __forceinline__ void store_row(TI* p, const RowMap& m, const float v[8]) {
  if (!m.on) return;
  if constexpr (HALF) {
    IO<TI>::store4(p + m.o1, v);
    IO<TI>::store4(p + m.o2, v + 4);
  } else if constexpr (sizeof(TI) == 2) {
    bf16x8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = (bf16)v[e];
    *reinterpret_cast<bf16x8*>(p + m.o1) = r;
  } else {
    IO<TI>::store4(p + m.o1, v);
    IO<TI>::store4(p + m.o2, v + 4);
  }
}

__device__ __forceinline__ void load_weight(const float* w, const RowMap& m, float v[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = w && m.on ? w[m.o1 + e] : 1.f;
    v[4 + e] = w && m.on ? w[m.o2 + e] : 1.f;
  }
}

// The lane's 4 pairs turned by (c, s); sign -1: turned back.
template <bool HALF>
__device__ __forceinline__ void rotate(float v[8], const float c[4], const float s[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ia = HALF ? i : 2 * i, ib = HALF ? 4 + i : 2 * i + 1;
    const float x = v[ia], y = v[ib];
    v[ia] = __builtin_fmaf(x, c[i], -y * s[i]);
    v[ib] = __builtin_fmaf(y, c[i], x * s[i]);
  }
}

// The 4 angles of a lane at position pos; lanes that rotate nothing get the identity.
__device__ __forceinline__ void lane_angles(const RopeArgs& a, const RowMap& m, int j, int64_t t, float back,
                                            float c[4], float s[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (!m.rot) return;
  const int pos = a.pos[t];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    turn_cs(pos, a.freq[4 * j + i], c[i], s[i]);
    c[i] *= a.mag;
    s[i] *= a.mag * back;
  }
}

template <typename TI, int LPR, bool HALF>
__global__ __launch_bounds__(256) void k_rope_fwd(RopeArgs a) {
  constexpr int GPB = 256 / LPR;
  const int j = threadIdx.x % LPR;
  const int64_t t = (int64_t)blockIdx.x * GPB + threadIdx.x / LPR;
  if (t >= a.T) return;
  const RowMap m = row_map<HALF>(j, a.D, a.RD);
  float c[4], s[4];
  lane_angles(a, m, j, t, 1.f, c, s);
  const int heads = a.hq + a.hk, h0 = blockIdx.y * a.hc, h1 = min(h0 + a.hc, heads);
  const float mean = a.norm == 2 ? 1.f / a.D : 1.f;
  const auto run = [&](const TI* x, TI* y, const float* w, int lo, int hi) {
    if (lo >= hi) return;
    float wt[8];
    load_weight(w, m, wt);
    for (int h = lo; h < hi; ++h) {
      float v[8];
      load_row<TI, HALF>(x + (int64_t)h * a.D, m, v);
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
        const float r = 1.f / sqrtf(__builtin_fmaf(group_sum<LPR>(ss), mean, a.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r * wt[e];
      }
      if (m.rot) rotate<HALF>(v, c, s);
      store_row<TI, HALF>(y + (int64_t)h * a.D, m, v);
    }
  };
  run((const TI*)a.q + t * a.qs, (TI*)a.qo + t * a.qos, a.wq, h0, min(h1, a.hq));
  run((const TI*)a.k + t * a.ks, (TI*)a.ko + t * a.kos, a.wk, max(h0 - a.hq, 0), h1 - a.hq);
}

template <typename TI, int LPR, bool HALF>
__global__ __launch_bounds__(256) void k_rope_bwd(RopeArgs a) {
  constexpr int GPB = 256 / LPR;
  __shared__ float red[256][17];
  const int j = threadIdx.x % LPR;
  const RowMap m = row_map<HALF>(j, a.D, a.RD);
  const int heads = a.hq + a.hk, h0 = blockIdx.y * a.hc, h1 = min(h0 + a.hc, heads);
  const float mean = a.norm == 2 ? 1.f / a.D : 1.f;
  float acc[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[0][e] = acc[1][e] = 0.f;
  for (int64_t t = (int64_t)blockIdx.x * GPB + threadIdx.x / LPR; t < a.T; t += (int64_t)gridDim.x * GPB) {
    float c[4], s[4];
    lane_angles(a, m, j, t, -1.f, c, s);
    const auto run = [&](const TI* x, const TI* dy, TI* dx, const float* w, float sum[8], int lo, int hi) {
      if (lo >= hi) return;
      float wt[8];
      load_weight(w, m, wt);
      for (int h = lo; h < hi; ++h) {
        float g[8];
        load_row<TI, HALF>(dy + (int64_t)h * a.D, m, g);
        if (m.rot) rotate<HALF>(g, c, s);
        if (a.norm) {
          float v[8];
          load_row<TI, HALF>(x + (int64_t)h * a.D, m, v);
          float ss = 0.f, vg = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = __builtin_fmaf(v[e], v[e], ss);
            vg = __builtin_fmaf(v[e], g[e] * wt[e], vg);
          }
          const float r = 1.f / sqrtf(__builtin_fmaf(group_sum<LPR>(ss), mean, a.eps));
          const float k = group_sum<LPR>(vg) * r * r * mean; // c (n . dn) / |x's scale|
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            sum[e] = __builtin_fmaf(g[e], v[e] * r, sum[e]);
            g[e] = r * (g[e] * wt[e] - k * v[e]);
          }
        }
        store_row<TI, HALF>(dx + (int64_t)h * a.D, m, g);
      }
    };
    run((const TI*)a.q + t * a.qs, (const TI*)a.dqo + t * a.qos, (TI*)a.dq + t * a.dqs, a.wq, acc[0], h0,
        min(h1, a.hq));
    run((const TI*)a.k + t * a.ks, (const TI*)a.dko + t * a.kos, (TI*)a.dk + t * a.dks, a.wk, acc[1],
        max(h0 - a.hq, 0), h1 - a.hq);
  }
  if (!a.dwq && !a.dwk) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    red[threadIdx.x][e] = acc[0][e];
    red[threadIdx.x][8 + e] = acc[1][e];
  }
  __syncthreads();
  float* part = a.part + ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.D;
  for (int i = threadIdx.x; i < LPR * 16; i += 256) {
    const int jj = i / 16, e = i % 16;
    const RowMap mm = row_map<HALF>(jj, a.D, a.RD);
    if (!mm.on) continue;
    float x = 0.f;
#pragma unroll
    for (int g = 0; g < GPB; ++g) x += red[g * LPR + jj][e];
    const int ee = e & 7;
    part[(e >> 3) * a.D + (ee < 4 ? mm.o1 + ee : mm.o2 + ee - 4)] = x;
  }
}

// dq_weight and dk_weight: the workgroups' partial sums, added in a fixed order: 16 columns a
// workgroup, 16 slices of the rows each, then the slices.
__global__ __launch_bounds__(256) void k_rope_reduce(RopeArgs a, int blocks) {
  __shared__ float red[16][17];
  const int c = threadIdx.x & 15, s = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;
  float x = 0.f;
  if (col < 2 * a.D)
    for (int b = s; b < blocks; b += 16) x += a.part[(size_t)b * 2 * a.D + col];
  red[s][c] = x;
  __syncthreads();
  if (s == 0 && col < 2 * a.D) {
    x = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x += red[i][c];
    if (col < a.D) {
      if (a.dwq) a.dwq[col] = x;
    } else if (a.dwk) {
      a.dwk[col - a.D] = x;
    }
  }
}

static int lanes_of(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Heads per unit of work: all of a token's heads share one set of cosines and sines, but a short
// call is cut further, down to one head, to keep 2048 waves.
static int heads_per_unit(int64_t T, int heads, int D) {
  const int64_t want = 2048 * (64 / lanes_of(D));
  int64_t hc = (T * heads + want - 1) / want;
  return (int)(hc < 1 ? 1 : hc > heads ? heads : hc);
}

static dim3 bwd_grid(int64_t T, int heads, int D) {
  const int gpb = 256 / lanes_of(D), hc = heads_per_unit(T, heads, D);
  int64_t x = (T + gpb - 1) / gpb;
  if (x > 1024) x = 1024;
  return dim3((unsigned)(x < 1 ? 1 : x), (heads + hc - 1) / hc);
}

int rope_bwd_blocks(int64_t T, int heads, int D) {
  const dim3 g = bwd_grid(T, heads, D);
  return (int)(g.x * g.y);
}

template <typename TI, int LPR>
static int rope_fwd_t(RopeArgs a, hipStream_t s) {
  const int heads = a.hq + a.hk;
  a.hc = heads_per_unit(a.T, heads, a.D);
  const dim3 grid((unsigned)((a.T + 256 / LPR - 1) / (256 / LPR)), (heads + a.hc - 1) / a.hc);
  if (a.interleaved) hipLaunchKernelGGL((k_rope_fwd<TI, LPR, false>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_rope_fwd<TI, LPR, true>), grid, dim3(256), 0, s, a);
  return (int)hipGetLastError();
}

template <typename TI, int LPR>
static int rope_bwd_t(RopeArgs a, hipStream_t s) {
  const int heads = a.hq + a.hk;
  a.hc = heads_per_unit(a.T, heads, a.D);
  const dim3 grid = bwd_grid(a.T, heads, a.D);
  if (a.interleaved) hipLaunchKernelGGL((k_rope_bwd<TI, LPR, false>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_rope_bwd<TI, LPR, true>), grid, dim3(256), 0, s, a);
  const int e = (int)hipGetLastError();
  if (e || (!a.dwq && !a.dwk)) return e;
  hipLaunchKernelGGL(k_rope_reduce, dim3((2 * a.D + 15) / 16), dim3(256), 0, s, a, (int)(grid.x * grid.y));
  return (int)hipGetLastError();
}

int launch_rope_fwd(const RopeArgs& a, int dtype, void* stream) {
  if (a.T == 0) return 0;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (lanes_of(a.D) + (dtype == 0 ? 0 : 1)) {
    case 8: return rope_fwd_t<bf16, 8>(a, s);
    case 9: return rope_fwd_t<float, 8>(a, s);
    case 16: return rope_fwd_t<bf16, 16>(a, s);
    case 17: return rope_fwd_t<float, 16>(a, s);
    case 32: return rope_fwd_t<bf16, 32>(a, s);
    default: return rope_fwd_t<float, 32>(a, s);
  }
}

int launch_rope_bwd(const RopeArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (a.T == 0) { // no tokens: the weight gradients are zero
    if (!a.dwq && !a.dwk) return 0;
    hipLaunchKernelGGL(k_rope_reduce, dim3((2 * a.D + 15) / 16), dim3(256), 0, s, a, 0);
    return (int)hipGetLastError();
  }
  switch (lanes_of(a.D) + (dtype == 0 ? 0 : 1)) {
    case 8: return rope_bwd_t<bf16, 8>(a, s);
    case 9: return rope_bwd_t<float, 8>(a, s);
    case 16: return rope_bwd_t<bf16, 16>(a, s);
    case 17: return rope_bwd_t<float, 16>(a, s);
    case 32: return rope_bwd_t<bf16, 32>(a, s);
    default: return rope_bwd_t<float, 32>(a, s);
  }
}

} // namespace gdn
