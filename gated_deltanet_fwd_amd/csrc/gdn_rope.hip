// Norms of the q and k heads with the position rotation, forward and backward (gfx950). Per head
// row x of a token at position p, c = 1/D (RMS) or 1 (L2), r = 1/sqrt(c sum x^2 + eps):
//
//   n = x r,  z = n w,  y = m R(p f) z           (R turns the pairs of the first RD values)
//   dz = m R(-p f) dy,  dn = dz w,  dw = sum dz n,  dx = r (dn - c n (n.dn))
//
// A row is held by 8, 16 or 32 lanes, 8 values a lane: 4 consecutive ones of each half of the
// rotated part (or of the part that passes), so that both values of a pair are in one lane in both
// layouts. A wave takes a token's q or its k heads (or some of them) and goes through their rows, 512
// values a pass, so the lanes of an access lie next to each other (with the rows of 4 tokens in one
// access 32,768 tokens of 16 + 16 heads moved 3.9 TB/s instead of 5.5). The next pass's rows are
// loaded while one is computed. What bounds both directions is memory.
//
// The angle is exact: a frequency is a 64-bit fraction of a turn per position, and the product with
// the position modulo 2^64 drops whole turns. Its top 32 bits give the quadrant and a remainder of
// at most 1/8 turn, where the Taylor polynomials of sine and cosine to x^9 and x^10 are off by less
// than 2e-9 and 2e-10.
#include <algorithm>

#include "gdn_device.h"

namespace gdn {

// Waves that a short call is cut into, and that a long one has at most (see rope_shape).
constexpr int64_t FWD_FILL = 8192, FWD_MOST = 32768, BWD_FILL = 4096, BWD_MOST = 4096;

template <int CTRL>
__device__ __forceinline__ float dpp_of(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// Sum over a row's LPR lanes, in every lane.
template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
  x += dpp_of<0xB1>(x);  // lane ^ 1
  x += dpp_of<0x4E>(x);  // lane ^ 2
  x += dpp_of<0x141>(x); // 7 - lane within 8: the other quad
  if constexpr (LPR >= 16) x += dpp_of<0x140>(x); // 15 - lane within 16
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

// Where a lane's 8 values lie in a row: values 0..3 at o1, 4..7 at o2, and the indices of its four
// pairs' frequencies: f1, f1 + 1 and f2, f2 + 1.
struct RowMap {
  int o1, o2, f1, f2;
  bool on, rot;
};
template <bool HALF>
__device__ __forceinline__ RowMap row_map(int j, int D, int RD) {
  RowMap m;
  m.on = 8 * j < D;
  m.rot = 8 * j < RD;
  const int k = m.rot ? j : j - RD / 8, from = m.rot ? 0 : RD, size = m.rot ? RD : D - RD;
  m.o1 = from + 4 * k;
  m.o2 = m.o1 + size / 2;
  m.f1 = HALF ? 4 * j : 2 * j;
  m.f2 = HALF ? 4 * j + 2 : RD / 4 + 2 * j;
  return m;
}

// A lane's 8 values as they are stored.
template <typename TI>
struct Raw {
  typedef TI vec __attribute__((ext_vector_type(4)));
  vec a, b;
  __device__ __forceinline__ void load(const TI* p, const RowMap& m) { // lanes past the row: its first values
    a = *reinterpret_cast<const vec*>(p + (m.on ? m.o1 : 0));
    b = *reinterpret_cast<const vec*>(p + (m.on ? m.o2 : 4));
  }
  __device__ __forceinline__ void unpack(float v[8], bool on) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = on ? (float)a[e] : 0.f;
      v[4 + e] = on ? (float)b[e] : 0.f;
    }
  }
};

template <typename TI>
__device__ __forceinline__ void store_row(TI* p, const RowMap& m, const float v[8]) {
  IO<TI>::store4(p + m.o1, v);
  IO<TI>::store4(p + m.o2, v + 4);
}

// The lane's 4 pairs turned by (c, s).
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

// x of the lanes with the same lane % 16 (rows 0..3) or lane % 32 (rows 0, 1), in every lane. The
// lane swaps exchange x's odd 16-lane rows (or its upper half) with y's even ones; the copies keep
// the compiler from folding a swap of one value with itself away.
__device__ __forceinline__ void gather_rows(float x, float out[4]) {
  unsigned a = __builtin_bit_cast(unsigned, x), b = a;
  asm("" : "+v"(b));
  const auto s = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  unsigned e = s[0], e2 = s[0], o = s[1], o2 = s[1];
  asm("" : "+v"(e2), "+v"(o2));
  const auto p = __builtin_amdgcn_permlane32_swap(e, e2, false, false), q = __builtin_amdgcn_permlane32_swap(o, o2, false, false);
  out[0] = __builtin_bit_cast(float, (unsigned)p[0]);
  out[1] = __builtin_bit_cast(float, (unsigned)q[0]);
  out[2] = __builtin_bit_cast(float, (unsigned)p[1]);
  out[3] = __builtin_bit_cast(float, (unsigned)q[1]);
}
__device__ __forceinline__ void gather_halves(float x, float out[2]) {
  unsigned a = __builtin_bit_cast(unsigned, x), b = a;
  asm("" : "+v"(b));
  const auto s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  out[0] = __builtin_bit_cast(float, (unsigned)s[0]);
  out[1] = __builtin_bit_cast(float, (unsigned)s[1]);
}

// A lane's frequencies and angles. Where a pass holds one token, the lanes that share the four pairs
// of position j divide them (one each of four lane rows, or two each of two halves) and exchange the
// cosines and sines; where it holds several, each lane makes its four.
template <int LPR>
__device__ __forceinline__ void lane_freqs(const RopeArgs& a, const RowMap& m, bool one, uint64_t f[4]) {
  f[0] = f[1] = f[2] = f[3] = 0;
  if (!m.rot) return;
  const int lane = threadIdx.x & 63;
  if (!one) {
    f[0] = a.freq[m.f1];
    f[1] = a.freq[m.f1 + 1];
    f[2] = a.freq[m.f2];
    f[3] = a.freq[m.f2 + 1];
  } else if constexpr (LPR <= 16) {
    const int i = lane >> 4;
    f[0] = a.freq[(i < 2 ? m.f1 : m.f2) + (i & 1)];
  } else {
    const int at = lane < 32 ? m.f1 : m.f2;
    f[0] = a.freq[at];
    f[1] = a.freq[at + 1];
  }
}

// The lane's 4 angles at position pos (lanes that rotate nothing get values that are not used).
template <int LPR>
__device__ __forceinline__ void lane_angles(const RopeArgs& a, const uint64_t f[4], bool one, int pos, float back,
                                            float c[4], float s[4]) {
  float x, y;
  if (!one) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn_cs(pos, f[i], x, y);
      c[i] = x * a.mag;
      s[i] = y * a.mag * back;
    }
    return;
  }
  turn_cs(pos, f[0], x, y);
  if constexpr (LPR <= 16) {
    gather_rows(x * a.mag, c);
    gather_rows(y * a.mag * back, s);
  } else {
    float t[2], u[2];
    gather_halves(x * a.mag, t);
    gather_halves(y * a.mag * back, u);
    c[0] = t[0], c[2] = t[1], s[0] = u[0], s[2] = u[1];
    turn_cs(pos, f[1], x, y);
    gather_halves(x * a.mag, t);
    gather_halves(y * a.mag * back, u);
    c[1] = t[0], c[3] = t[1], s[1] = u[0], s[3] = u[1];
  }
}

__device__ __forceinline__ void load_weight(const float* w, const RowMap& m, float v[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 1.f;
  if (!w || !m.on) return;
  const f32x4 x = *reinterpret_cast<const f32x4*>(w + m.o1), y = *reinterpret_cast<const f32x4*>(w + m.o2);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = x[e], v[4 + e] = y[e];
}

// A wave's work: passes [p0, p1) over the rows of the token groups t, t + dt, ... of its side. A pass
// takes 64 / LPR rows: of one token, or with fewer heads than that, the heads of `tpp` tokens
// (lane group g then holds head `head` of the group's token `tok`).
struct Share {
  int t, dt, p0, p1, groups, head, tok;
};
template <int LPR>
__device__ __forceinline__ Share share_of(const RopeArgs& a, const RopeSide& s, int block) {
  const int wave = block * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = wave % s.chunks, g = (threadIdx.x & 63) / LPR;
  Share sh;
  sh.t = wave / s.chunks;
  sh.dt = s.blocks * 4 / s.chunks;
  sh.p0 = c * s.per;
  sh.p1 = min(sh.p0 + s.per, s.passes);
  sh.groups = (a.T - 1) / s.tpp + 1;
  sh.head = g & ((64 / LPR / s.tpp) - 1);
  sh.tok = g / (64 / LPR / s.tpp);
  return sh;
}
// A lane's row in pass i over token group t, from the start of the group's first token: offsets
// inside a group are 32-bit (the host checks the strides); rows and tokens past the end are cut.
template <int LPR>
__device__ __forceinline__ int row_at(const RopeArgs& a, const RopeSide& s, const Share& sh, int t, int i, int64_t stride) {
  return min(sh.tok, a.T - 1 - t * s.tpp) * (int)stride + min(i * (64 / LPR) + sh.head, s.heads - 1) * a.D;
}
__device__ __forceinline__ int pos_at(const RopeArgs& a, const RopeSide& s, const Share& sh, int t) {
  return a.RD ? a.pos[min(t * s.tpp + sh.tok, a.T - 1)] : 0;
}

template <typename TI, int LPR, bool HALF>
__global__ __launch_bounds__(256) void k_rope_fwd(RopeArgs a) {
  constexpr int RPW = 64 / LPR;
  const int side = (int)blockIdx.x >= a.side[0].blocks;
  const RopeSide sd = a.side[side];
  Share sh = share_of<LPR>(a, sd, blockIdx.x - (side ? a.side[0].blocks : 0));
  if (sh.t >= sh.groups) return;
  const RowMap m = row_map<HALF>((threadIdx.x & 63) % LPR, a.D, a.RD);
  const auto load = [&](Raw<TI>& r, int t, int i) {
    r.load((const TI*)sd.x + (int64_t)t * sd.tpp * sd.xs + row_at<LPR>(a, sd, sh, t, i, sd.xs), m);
  };
  Raw<TI> cur, next;
  load(cur, sh.t, sh.p0);
  int pos = pos_at(a, sd, sh, sh.t);
  const bool one = sd.tpp == 1;
  uint64_t f[4];
  lane_freqs<LPR>(a, m, one, f);
  float w[8];
  load_weight(sd.w, m, w);
  const float mean = a.norm == 2 ? 1.f / a.D : 1.f;
  for (; sh.t < sh.groups; sh.t += sh.dt) {
    const int tn = min(sh.t + sh.dt, sh.groups - 1);
    float c[4], s[4];
    lane_angles<LPR>(a, f, one, pos, 1.f, c, s);
    pos = pos_at(a, sd, sh, tn);
    for (int i = sh.p0; i < sh.p1; ++i) {
      const bool more = i + 1 < sh.p1;
      load(next, more ? sh.t : tn, more ? i + 1 : sh.p0);
      float v[8];
      cur.unpack(v, m.on);
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
        const float r = inv_sqrt_any(__builtin_fmaf(group_sum<LPR>(ss), mean, a.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r * w[e];
      }
      if (m.rot) rotate<HALF>(v, c, s);
      if (m.on && i * RPW + sh.head < sd.heads && sh.t * sd.tpp + sh.tok < a.T)
        store_row((TI*)sd.out + (int64_t)sh.t * sd.tpp * sd.outs + row_at<LPR>(a, sd, sh, sh.t, i, sd.outs), m, v);
      cur = next;
    }
  }
}

// The weight's gradient is summed in the lane over all its rows, then over the workgroup's lanes in
// LDS, and over the side's workgroups by k_rope_reduce. (A row that is loaded ahead and not this
// wave's to compute may be written in place meanwhile: nothing made of it is kept.)
template <typename TI, int LPR, bool HALF>
__global__ __launch_bounds__(256) void k_rope_bwd(RopeArgs a) {
  constexpr int RPW = 64 / LPR, GPB = 256 / LPR;
  __shared__ float red[256][9];
  const int side = (int)blockIdx.x >= a.side[0].blocks;
  const RopeSide sd = a.side[side];
  Share sh = share_of<LPR>(a, sd, blockIdx.x - (side ? a.side[0].blocks : 0));
  const RowMap m = row_map<HALF>((threadIdx.x & 63) % LPR, a.D, a.RD);
  const auto load = [&](Raw<TI>& x, Raw<TI>& d, int t, int i) {
    d.load((const TI*)sd.dy + (int64_t)t * sd.tpp * sd.dys + row_at<LPR>(a, sd, sh, t, i, sd.dys), m);
    if (a.norm) x.load((const TI*)sd.x + (int64_t)t * sd.tpp * sd.xs + row_at<LPR>(a, sd, sh, t, i, sd.xs), m);
  };
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  if (sh.t < sh.groups) {
    Raw<TI> cx, cd, nx, nd;
    load(cx, cd, sh.t, sh.p0);
    int pos = pos_at(a, sd, sh, sh.t);
    const bool one = sd.tpp == 1;
    uint64_t f[4];
    lane_freqs<LPR>(a, m, one, f);
    float w[8];
    load_weight(sd.w, m, w);
    const float mean = a.norm == 2 ? 1.f / a.D : 1.f;
    for (; sh.t < sh.groups; sh.t += sh.dt) {
      const int tn = min(sh.t + sh.dt, sh.groups - 1);
      float c[4], s[4];
      lane_angles<LPR>(a, f, one, pos, -1.f, c, s);
      pos = pos_at(a, sd, sh, tn);
      for (int i = sh.p0; i < sh.p1; ++i) {
        const bool more = i + 1 < sh.p1;
        load(nx, nd, more ? sh.t : tn, more ? i + 1 : sh.p0);
        const bool mine = i * RPW + sh.head < sd.heads && sh.t * sd.tpp + sh.tok < a.T;
        float d[8];
        cd.unpack(d, m.on);
        if (m.rot) rotate<HALF>(d, c, s);
        if (a.norm) {
          float v[8], dn[8], ss = 0.f, vd = 0.f;
          cx.unpack(v, m.on);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dn[e] = d[e] * w[e];
            ss = __builtin_fmaf(v[e], v[e], ss);
            vd = __builtin_fmaf(v[e], dn[e], vd);
          }
          const float r = inv_sqrt_any(__builtin_fmaf(group_sum<LPR>(ss), mean, a.eps));
          const float k = group_sum<LPR>(vd) * r * mean; // (r^3 overflows for rows that dx = r (dn - k n) fits)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float n = v[e] * r;
            sum[e] = mine ? __builtin_fmaf(d[e], n, sum[e]) : sum[e];
            d[e] = r * __builtin_fmaf(-k, n, dn[e]);
          }
        }
        if (m.on && mine)
          store_row((TI*)sd.out + (int64_t)sh.t * sd.tpp * sd.outs + row_at<LPR>(a, sd, sh, sh.t, i, sd.outs), m, d);
        cx = nx;
        cd = nd;
      }
    }
  }
  if (!sd.dw) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[threadIdx.x][e] = sum[e];
  __syncthreads();
  if (threadIdx.x < LPR * 8) {
    const int jj = threadIdx.x / 8, e = threadIdx.x % 8;
    const RowMap mm = row_map<HALF>(jj, a.D, a.RD);
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < GPB; ++k) x += red[k * LPR + jj][e];
    if (mm.on) a.part[(size_t)blockIdx.x * a.D + (e < 4 ? mm.o1 + e : mm.o2 + e - 4)] = x;
  }
}

// dq_weight and dk_weight: the workgroups' partial sums, added in a fixed order: 8 columns a
// workgroup, 128 slices of the rows each, then the slices, 8 by 8 and the 16 sums of those.
__global__ __launch_bounds__(1024) void k_rope_reduce(RopeArgs a) {
  __shared__ float red[128][9];
  const int c = threadIdx.x & 7, s = threadIdx.x >> 3, side = blockIdx.x * 8 >= a.D;
  const int col = blockIdx.x * 8 + c - (side ? a.D : 0);
  const int b0 = side ? a.side[0].blocks : 0, b1 = b0 + a.side[side].blocks;
  float* dw = a.side[side].dw;
  if (!dw) return;
  float x = 0.f;
#pragma unroll 8
  for (int b = b0 + s; b < b1; b += 128) x += a.part[(size_t)b * a.D + col];
  red[s][c] = x;
  __syncthreads();
  if (s < 16) {
    x = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x += red[8 * s + i][c];
  }
  __syncthreads();
  if (s < 16) red[s][c] = x;
  __syncthreads();
  if (s != 0) return;
  x = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) x += red[i][c];
  dw[col] = x;
}

static int lanes_of(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// The grid of a side. A wave takes a token group's passes in turn, loading one ahead. Short calls are
// cut to `fill` waves over both sides, down to one pass a wave: 4096 tokens of 16 + 16 heads, 128
// wide, forward, take 12.8 us in 8192 waves, 17 us in 32768, each with its own cosines and sines.
// Long ones go over the groups with up to `most`, each wave the same number of groups: 32,768 such
// tokens take 97 us in 32768 waves, 101 us in 8192; backward, where each workgroup leaves a row of
// partial sums, 154 us in 4096 and 159 us in 8192 or more. A backward without weights has the same limit:
// there more waves gain or lose by the sizes (4096 / 8192 / 32768 waves: 32,768 tokens, L2 150 / 150 / 144
// us, the rotation alone 96 / 98 / 93; 65,536 tokens of 3 + 1 heads, the rotation alone 32 / 30 / 32).
static void shape_side(RopeSide& s, int64_t T, int D, int all_heads, int64_t fill, int64_t most) {
  const int rpw = 64 / lanes_of(D);
  s.tpp = 1;
  while (s.heads > 0 && s.heads * s.tpp * 2 <= rpw) s.tpp *= 2;
  s.passes = (s.heads * s.tpp + rpw - 1) / rpw;
  s.per = s.passes;
  s.chunks = 1;
  s.blocks = 0;
  if (T == 0 || s.heads == 0) return;
  const int64_t groups = (T + s.tpp - 1) / s.tpp;
  fill = fill * s.heads / all_heads;
  most = std::max<int64_t>(most * s.heads / all_heads, 1);
  if (groups < fill) {
    const int64_t c = (fill + groups - 1) / groups;
    s.per = (int)(c >= s.passes ? 1 : (s.passes + c - 1) / c);
    s.chunks = (s.passes + s.per - 1) / s.per;
  }
  const int64_t each = std::max<int64_t>((groups + most / 2) / most, 1); // groups a wave
  const int64_t waves = (groups + each - 1) / each * s.chunks;
  // a whole number of token groups a step, so that a wave keeps its place in them
  s.blocks = (int)((waves + 4 * s.chunks - 1) / (4 * s.chunks)) * s.chunks;
}
void rope_shape(RopeArgs& a, bool bwd) {
  for (RopeSide& s : a.side)
    shape_side(s, a.T, a.D, a.side[0].heads + a.side[1].heads, bwd ? BWD_FILL : FWD_FILL, bwd ? BWD_MOST : FWD_MOST);
}

template <typename TI, int LPR>
static int rope_t(const RopeArgs& a, bool bwd, hipStream_t s) {
  const dim3 grid((unsigned)(a.side[0].blocks + a.side[1].blocks)), blk(256);
  if (bwd) {
    if (a.interleaved) hipLaunchKernelGGL((k_rope_bwd<TI, LPR, false>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((k_rope_bwd<TI, LPR, true>), grid, blk, 0, s, a);
  } else {
    if (a.interleaved) hipLaunchKernelGGL((k_rope_fwd<TI, LPR, false>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((k_rope_fwd<TI, LPR, true>), grid, blk, 0, s, a);
  }
  return (int)hipGetLastError();
}

int launch_rope(const RopeArgs& a, bool bwd, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  int e = 0;
  if (a.T > 0) {
    switch (lanes_of(a.D) + (dtype == 0 ? 0 : 1)) {
      case 8: e = rope_t<bf16, 8>(a, bwd, s); break;
      case 9: e = rope_t<float, 8>(a, bwd, s); break;
      case 16: e = rope_t<bf16, 16>(a, bwd, s); break;
      case 17: e = rope_t<float, 16>(a, bwd, s); break;
      case 32: e = rope_t<bf16, 32>(a, bwd, s); break;
      default: e = rope_t<float, 32>(a, bwd, s); break;
    }
  }
  if (e || (!a.side[0].dw && !a.side[1].dw)) return e;
  hipLaunchKernelGGL(k_rope_reduce, dim3(2 * a.D / 8), dim3(1024), 0, s, a); // no tokens: zeros
  return (int)hipGetLastError();
}

} // namespace gdn
