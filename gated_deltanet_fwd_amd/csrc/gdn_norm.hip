// RMS norm of rows of d values with the residual's addition, forward (to the io type, or to 8 bits with scales) and
// backward (gfx950). With x' = x + r in FP32 (x without a residual):
//
//   y = w x' / sqrt(mean(x'^2) + eps),   residual_out = x'
//   dn = w dy, n = x' / sqrt(..):   dx = (dn - n mean(n dn)) / sqrt(..) + d_residual,   dw = sum over rows of dy n
//
// It costs moving the rows once: 32,768 rows of 2048 bf16 values with residual to 8 bits, 472 MB in 85 us (5.6 TB/s),
// backward 537 MB in 104 us (5.2 TB/s; the sum of dw's parts 4.5 of them). LANES lanes take a row, 8 neighbouring
// values a lane and pass, and keep it in registers between the sum and its use.
#include <algorithm>

#include "gdn_device.h"

namespace gdn {

// Sum over the LANES lanes of a row, in every lane. tmp: one float a wave.
template <int LANES>
__device__ __forceinline__ float row_total(float x, float* tmp) {
  x = col_sum4(row_sum16(x));
  if constexpr (LANES > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / 64; ++i) x += tmp[i];
  }
  return x;
}
__device__ __forceinline__ unsigned larger(unsigned x, int lanes) { return max(x, (unsigned)__shfl_xor((int)x, lanes)); }
template <int LANES>
__device__ __forceinline__ unsigned row_largest(unsigned x, unsigned* tmp) {
#pragma unroll
  for (int by = 1; by < 64; by *= 2) x = larger(x, by);
  if constexpr (LANES > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < LANES / 64; ++i) x = max(x, tmp[i]);
  }
  return x;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float v[8]) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    IO<float>::store4((float*)p, v);
    IO<float>::store4((float*)p + 4, v + 4);
  }
}

// 8 values as e4m3 (round to nearest even; they are at most 448 but for the scale's rounding, which rounds back)
__device__ __forceinline__ uint2 to_e4m3(const float v[8]) {
  int a = 0, b = 0;
  a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], a, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], b, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
  return make_uint2((unsigned)a, (unsigned)b);
}

// The scale of values whose largest magnitude has the bits `most` (as integers these order magnitudes, NaN
// above infinity, so a NaN is not lost): most / 448, 1 for zeros, and no less than the smallest normal number, whose
// inverse is still one. The product with 1 / 448 and its remainder give the nearest quotient (all mantissas were tried).
__device__ __forceinline__ float scale_of(unsigned most) {
  constexpr float INV = 1.f / 448.f;
  const float x = __builtin_bit_cast(float, most), q = x * INV, s = __builtin_fmaf(__builtin_fmaf(-q, 448.f, x), INV, q);
  if (most == 0) return 1.f;
  return most >= 0x7f800000u ? x : s < 0x1p-126f ? 0x1p-126f : s;
}

// v / scale for a rounding to 8 bits, which takes it to where it would take the quotient itself: q is brought within a
// step of the quotient by its remainder, and where the remainder that is left says that the quotient is not q, an even q
// goes one step towards it: midpoints of two 8-bit values are even, so that no value lies on one by rounding (as FP32's nearest
// quotient can). Remainders are exact from scales of 2^-90 on. `by`: scale, 0 where that is infinite (finite / infinite
// is 0 and leaves no remainder).
__device__ __forceinline__ float quotient(float v, float by, float inv) {
  float q = v * inv;
  q = __builtin_fmaf(__builtin_fmaf(-q, by, v), inv, q);
  const float left = __builtin_fmaf(-q, by, v);
  const int bits = __builtin_bit_cast(int, q), step = (__builtin_bit_cast(int, left) ^ bits) < 0 ? -1 : 1;
  return __builtin_bit_cast(float, left != 0.f && !(bits & 1) ? bits + step : bits);
}
// 8 values over their scale. v times the inverse (itself off by one step at most) is off by less than three, so that alone
// is right but where it lies that near to a midpoint (the low 20 bits of one are 0x80000), or below 2^-6, where 8-bit
// values and midpoints are spaced otherwise. With quotient() for all of them 32,768 rows of 2048 took 93 us instead
// of 87.
__device__ __forceinline__ void over_scale(float v[8], float scale) {
  const float inv = __builtin_amdgcn_rcpf(scale);
  float q[8], least = __builtin_inff();
  unsigned off = ~0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q[e] = v[e] * inv;
    off = min(off, (__builtin_bit_cast(unsigned, q[e]) << 12) + 0x80003000u);
    least = __builtin_fminf(least, __builtin_fabsf(q[e]));
  }
  if (off <= 0x6000u || least < 0x1p-6f) {
    const float by = scale < __builtin_inff() ? scale : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = quotient(v[e], by, inv);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = q[e];
}

template <typename T, int LANES, int NP>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void k_norm_fwd(NormArgs a) {
  constexpr int PER = LANES < 256 ? 256 / LANES : 1;
  __shared__ float tmp[LANES / 64 < 4 ? 4 : LANES / 64];
  const int lane = threadIdx.x % LANES;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * PER + threadIdx.x / LANES;
  if (row >= a.rows) return; // (LANES > 64: the whole workgroup)
  const T* x = (const T*)a.x + row * a.xs;
  float v[NP][8], sum = 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int c = 8 * (lane + LANES * p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[p][e] = 0.f;
    if (c < a.D) IO<T>::load8f(x + c, v[p]);
  }
  if (a.res) {
    const T* r = (const T*)a.res + row * a.rs;
    T* out = (T*)a.out + row * a.os;
    float u[NP][8];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = 8 * (lane + LANES * p);
      if (c < a.D) IO<T>::load8f(r + c, u[p]);
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = 8 * (lane + LANES * p);
      if (c < a.D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[p][e] += u[p][e];
        store8(out + c, v[p]);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(v[p][e], v[p][e], sum);
  const float r = inv_sqrt_any(row_total<LANES>(sum, tmp) / (float)a.D + a.eps);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int c = 8 * (lane + LANES * p);
    if (c < a.D) {
      float w[8];
      if (a.w) IO<float>::load8f(a.w + c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[p][e] = v[p][e] * r * (a.w ? w[e] : 1.f);
    }
  }
  if (!a.e4m3) {
    T* y = (T*)a.y + row * a.ys;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = 8 * (lane + LANES * p);
      if (c < a.D) store8(y + c, v[p]);
    }
    return;
  }
  uint8_t* y = (uint8_t*)a.y + row * a.ys;
  const bool whole = a.group == a.D;
  const int shift = whole ? 31 : 31 - __builtin_clz(a.group); // other groups are powers of two: which one a value is in
  float* scales = a.scales + row * (whole ? 1 : a.D >> shift);
  unsigned most[NP], all = 0;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    most[p] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) most[p] = max(most[p], __builtin_bit_cast(unsigned, v[p][e]) & 0x7fffffffu);
    all = max(all, most[p]);
  }
  if (whole) all = row_largest<LANES>(all, (unsigned*)tmp);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int c = 8 * (lane + LANES * p);
    unsigned m = all;
    if (!whole) { // 4, 8 or 16 neighbouring lanes
      m = larger(larger(most[p], 1), 2);
      if (a.group >= 64) m = larger(m, 4);
      if (a.group >= 128) m = larger(m, 8);
    }
    const float scale = scale_of(m);
    if (c < a.D) {
      over_scale(v[p], scale);
      *reinterpret_cast<uint2*>(y + c) = to_e4m3(v[p]);
      if ((c & (int)((1u << shift) - 1)) == 0) scales[c >> shift] = scale;
    }
  }
}

// Backward. A workgroup goes through rows PER at a time and sums its share of dw in registers; k_norm_dw adds
// the workgroups' in their order.
template <typename T, int LANES, int NP>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void k_norm_bwd(NormArgs a) {
  constexpr int PER = LANES < 256 ? 256 / LANES : 1;
  __shared__ float tmp[2][LANES / 64 < 4 ? 4 : LANES / 64];
  __shared__ float sums[PER > 1 ? PER * LANES * NP * 8 : 1];
  const int lane = threadIdx.x % LANES, own = threadIdx.x / LANES;
  float w[NP][8], dw[NP][8];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int c = 8 * (lane + LANES * p);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[p][e] = 1.f;
      dw[p][e] = 0.f;
    }
    if (a.w && c < a.D) IO<float>::load8f(a.w + c, w[p]);
  }
  for (int64_t row = (int64_t)blockIdx.x * PER + own; row < a.rows; row += (int64_t)gridDim.x * PER) {
    const T *x = (const T*)a.x + row * a.xs, *dy = (const T*)a.dy + row * a.ys;
    float n[NP][8], d[NP][8], res[NP][8], xx = 0.f, xd = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = 8 * (lane + LANES * p);
#pragma unroll
      for (int e = 0; e < 8; ++e) n[p][e] = d[p][e] = res[p][e] = 0.f;
      if (c < a.D) {
        IO<T>::load8f(x + c, n[p]);
        IO<T>::load8f(dy + c, d[p]);
        if (a.res) IO<T>::load8f((const T*)a.res + row * a.rs + c, res[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) xx = __builtin_fmaf(n[p][e], n[p][e], xx);
    const float r = inv_sqrt_any(row_total<LANES>(xx, tmp[0]) / (float)a.D + a.eps);
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[p][e] *= r;
        dw[p][e] = __builtin_fmaf(d[p][e], n[p][e], dw[p][e]);
        d[p][e] *= w[p][e];
        xd = __builtin_fmaf(n[p][e], d[p][e], xd);
      }
    const float m = row_total<LANES>(xd, tmp[1]) / (float)a.D;
    T* out = (T*)a.out + row * a.os;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = 8 * (lane + LANES * p);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[p][e] = __builtin_fmaf(r, __builtin_fmaf(-n[p][e], m, d[p][e]), res[p][e]);
      if (c < a.D) store8(out + c, d[p]);
    }
  }
  if (!a.dw) return;
  if constexpr (PER > 1) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int e = 0; e < 8; e += 4)
        *reinterpret_cast<float4*>(&sums[own * LANES * NP * 8 + 8 * (lane + LANES * p) + e]) = make_float4(dw[p][e], dw[p][e + 1], dw[p][e + 2], dw[p][e + 3]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += 256) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) s += sums[i * LANES * NP * 8 + c];
      a.part[(int64_t)blockIdx.x * a.D + c] = s;
    }
  } else {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = 8 * (lane + LANES * p);
      if (c < a.D) store8(a.part + (int64_t)blockIdx.x * a.D + c, dw[p]);
    }
  }
}

// dw[c] = sum over the workgroups' parts; 32 columns a workgroup, 32 rows of lanes (with 8 of them the sum of
// 1024 parts of 2048 values took 48 us, a chain of 128 loads)
__global__ __launch_bounds__(1024) void k_norm_dw(NormArgs a, int blocks) {
  __shared__ float s[32][33];
  const int x = threadIdx.x % 32, y = threadIdx.x / 32, c = blockIdx.x * 32 + x;
  float sum = 0.f;
  if (c < a.D) {
    constexpr int AHEAD = 8;
    for (int i = y; i < blocks; i += 32 * AHEAD) {
      float v[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) v[j] = i + 32 * j < blocks ? a.part[(int64_t)(i + 32 * j) * a.D + c] : 0.f;
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) sum += v[j];
    }
  }
  s[y][x] = sum;
  __syncthreads();
  sum = s[x][y]; // of column blockIdx.x 32 + y: a sum over 32 neighbouring lanes
#pragma unroll
  for (int by = 1; by < 32; by *= 2) sum += __shfl_xor(sum, by);
  if (x == 0 && blockIdx.x * 32 + y < (unsigned)a.D) a.dw[blockIdx.x * 32 + y] = sum;
}

// Lanes a row: a wave takes a short row, a workgroup a long one (us, bf16, forward with residual: 512 wide, 16,384 rows
// 10.0 by waves, 14.1 by workgroups, 1024 rows 2.9 and 3.1; 1024 wide 17.2 and 19.5, but 3.8 and 3.5 at 1024 rows;
// 2048 wide, 16,384 rows, 37 and 31. Backward, 1024 wide: 18.5 and 28.2, 5.3 and 5.6 at 128 rows).
static bool by_wave(const NormArgs& a, bool bwd) { return a.D <= 512 || (a.D <= 1024 && (bwd || a.rows > 1024)); }

// Workgroups of the backward: each leaves a row of sums to be added, and so takes four rows at least unless that would
// leave CUs idle (2048 wide, 1024 rows: 9.3 us; one row each 11.9), and many where there are many: 1024 of 256
// threads (2048 wide, 16,384 rows: 31 us, 512 43, 2048 35) or 512 of 1024 (16,384 wide: 257 us, 1024 274).
int norm_blocks(const NormArgs& a) {
  const int64_t four = (a.rows + 3) / 4, rows = by_wave(a, true) ? four : std::max(four, std::min<int64_t>(a.rows, 256));
  return (int)std::min<int64_t>(rows, a.D > 8192 ? 512 : 1024);
}

template <typename T, int LANES, int NP>
static int norm_t(const NormArgs& a, bool bwd, hipStream_t s) {
  constexpr int PER = LANES < 256 ? 256 / LANES : 1, THREADS = LANES > 256 ? LANES : 256;
  // one dimension of a launch holds less than 2^32 threads
  const int64_t blocks = (a.rows + PER - 1) / PER, x = blocks < (1 << 20) ? blocks : 1 << 20;
  if (!bwd) hipLaunchKernelGGL((k_norm_fwd<T, LANES, NP>), dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(THREADS), 0, s, a);
  else hipLaunchKernelGGL((k_norm_bwd<T, LANES, NP>), dim3((unsigned)norm_blocks(a)), dim3(THREADS), 0, s, a);
  return (int)hipGetLastError();
}
template <typename T>
static int norm_any(const NormArgs& a, bool bwd, hipStream_t s) {
  if (by_wave(a, bwd)) return a.D <= 512 ? norm_t<T, 64, 1>(a, bwd, s) : norm_t<T, 64, 2>(a, bwd, s);
  if (a.D <= 2048) return norm_t<T, 256, 1>(a, bwd, s);
  if (a.D <= 4096) return norm_t<T, 256, 2>(a, bwd, s);
  return a.D <= 8192 ? norm_t<T, 256, 4>(a, bwd, s) : norm_t<T, 1024, 2>(a, bwd, s);
}

int launch_norm_fwd(const NormArgs& a, int dtype, void* stream) {
  if (a.rows == 0) return 0;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == 0 ? norm_any<bf16>(a, false, s) : norm_any<float>(a, false, s);
}
int launch_norm_bwd(const NormArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (a.rows > 0)
    if (const int e = dtype == 0 ? norm_any<bf16>(a, true, s) : norm_any<float>(a, true, s)) return e;
  if (!a.dw) return 0;
  hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)((a.D + 31) / 32)), dim3(1024), 0, s, a, norm_blocks(a));
  return (int)hipGetLastError();
}

} // namespace gdn
