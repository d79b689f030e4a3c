// Linear attention with a decay for each head, chunked, forward and backward (gfx950). Per document and
// value head, a_t = exp(g_t):
//
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// One product carries everything. For rows a, b, c (d values each) of a document define, with G_t the sum
// of the log decays up to t and W the state it starts from,
//
//   forward:  y_t = sum_{s <= t} e^{G_t - G_s} (a_t.b_s) c_s + e^{G_t} a_t W      W <- e^{G_T} W + sum_s e^{G_T - G_s} b_s c_s^T
//   reverse:  y_t = sum_{s >= t} e^{G_s - G_t} (a_t.b_s) c_s + e^{G_T - G_t} a_t W  W <- e^{G_T} W + sum_s e^{G_s} b_s c_s^T
//
// Then with S the states from h0 and D their gradients from dht (D_t = a_{t+1} D_{t+1} + scale q_t do_t^T)
//
//   o  = scale forward(q, k, v; S),       dq = scale forward(do, v, k; S^T),
//   dk = reverse(v, do, scale q; D^T),    dv = reverse(k, scale q, do; D),
//   dg_t = sum_{s >= t} (q_s.dq_s - k_s.dk_s) + <ht, dht>
//
// (the last because scaling a_t scales what passes from before t to t and after, and nothing else).
//
// A document is cut into segments, each a workgroup a head: k_linear_states leaves what each segment adds
// to a state, k_linear_scan turns that into the states that segments start from, k_linear_walk goes through
// a segment in chunks of 64 tokens with the state in registers.
#include <atomic>

#include "gdn_device.h"

namespace gdn {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// ------------------------------------------------------------------------------------------------
// Operands of 16x16 products over 32 k values, in the k-permuted order of gdn_device.h: lane group g has the
// k values 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3. bf16 rows go to one instruction, f32 rows to eight of
// 4 k values (element e of every lane to the e-th), so both share all of the indexing.
template <typename T>
struct Op;
template <>
struct Op<bf16> {
  typedef bf16x8 frag;
  static constexpr int PADDED = 8; // elements of row padding in LDS
  // The terms that hold an FP32 value: 3 bf16 hold all of its 24 bits.
  static constexpr int EXACT = 3;
  static __device__ __forceinline__ frag along(const bf16* tile, int stride, int row, int k0) { return lds_kp(tile, stride, row, k0); }
  static __device__ __forceinline__ frag down(const bf16* tile, int stride, int k0, int m0) { return lds_tr_kp(tile, stride, k0, m0); }
  static __device__ __forceinline__ f32x4 mul(const frag& a, const frag& b, const f32x4& c) { return mfma(a, b, c); }
};
template <>
struct Op<float> {
  typedef f32x8 frag;
  static constexpr int PADDED = 4, EXACT = 1;
  static __device__ __forceinline__ frag along(const float* tile, int stride, int row, int k0) {
    const float* p = tile + row * stride + k0 + 4 * ((threadIdx.x & 63) >> 4);
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ frag down(const float* tile, int stride, int k0, int m0) {
    const float* p = tile + (k0 + 4 * ((threadIdx.x & 63) >> 4)) * stride + m0 + (threadIdx.x & 15);
    frag r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[e] = p[e * stride];
      r[4 + e] = p[(16 + e) * stride];
    }
    return r;
  }
  static __device__ __forceinline__ f32x4 mul(const frag& a, const frag& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
};

// FP32 values as NT operands whose sum they are: of bf16 each term takes the 8 leading bits of what the terms
// before it left.
template <typename T, int NT>
struct Terms {
  typename Op<T>::frag f[NT];
  __device__ __forceinline__ explicit Terms(const f32x8& x) {
    if constexpr (sizeof(T) == 4) {
      f[0] = x;
    } else {
      f32x8 left = x;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[n][e] = (bf16)left[e];
        if (n + 1 < NT) {
#pragma unroll
          for (int e = 0; e < 8; ++e) left[e] -= (float)f[n][e];
        }
      }
    }
  }
};
template <typename T, int NT>
__device__ __forceinline__ f32x4 mul_terms(const Terms<T, NT>& a, const typename Op<T>::frag& b, f32x4 c) {
#pragma unroll
  for (int n = NT - 1; n >= 0; --n) c = Op<T>::mul(a.f[n], b, c);
  return c;
}
template <typename T, int NT>
__device__ __forceinline__ f32x4 mul_terms(const typename Op<T>::frag& a, const Terms<T, NT>& b, f32x4 c) {
#pragma unroll
  for (int n = NT - 1; n >= 0; --n) c = Op<T>::mul(a, b.f[n], c);
  return c;
}
__device__ __forceinline__ f32x8 join(const f32x4& a, const f32x4& b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
template <typename T>
__device__ __forceinline__ f32x8 widen(const typename Op<T>::frag& x) {
  f32x8 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = (float)x[e];
  return r;
}

// ------------------------------------------------------------------------------------------------
// Segments. Document n's segments have the slots cu[n] / seg + n, + 1, ...: these do not meet (a document of l
// tokens has at most l / seg + 1 of them, rounded up, and the next document's first slot is at least that much
// further), so each workgroup finds its own by a search over cu_seqlens, and no table is made before. Values outside
// [0, T] or falling ones (which the caller must not give) are cut, so that every access stays inside the tensors.
struct Segment {
  int doc, i, t0, t1; // its document, its place there, its tokens
  bool live, first, last;
};
__device__ __forceinline__ int cut_to(int x, int T) { return min(max(x, 0), T); }
__device__ __forceinline__ int doc_slot(const LinearArgs& a, int n) { return a.seg == 0 ? n : cut_to(a.cu[n], a.T) / a.seg + n; }
__device__ __forceinline__ Segment find_segment(const LinearArgs& a, int slot) {
  int lo = 0, hi = a.N - 1; // the last document whose first slot is at most `slot`
  if (a.seg == 0) lo = slot;
  else
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (doc_slot(a, mid) <= slot) lo = mid;
      else hi = mid - 1;
    }
  Segment s;
  s.doc = lo;
  const int from = cut_to(a.cu[lo], a.T), to = max(cut_to(a.cu[lo + 1], a.T), from);
  s.i = a.seg == 0 ? 0 : slot - doc_slot(a, lo);
  const int64_t t0 = from + (int64_t)s.i * a.seg;
  s.live = s.i == 0 || (s.i > 0 && t0 < to);
  s.t0 = (int)(t0 < to ? t0 : to);
  s.t1 = a.seg == 0 ? to : (int)(t0 + a.seg < to ? t0 + a.seg : to);
  s.first = s.i == 0;
  s.last = s.t1 == to;
  return s;
}

// Workgroup -> (slot, value head). Workgroups go to the 8 XCDs in turn; the heads of one group, which read the
// same shared rows, are placed 8 apart and so on one XCD.
__device__ __forceinline__ bool place(const LinearArgs& a, int* slot, int* h) {
  const int b = blockIdx.x, per = 8 * a.G;
  const int sg = b / per, rem = b - sg * per;
  const int group = sg * 8 + (rem & 7);
  *slot = group / a.H;
  *h = (group - *slot * a.H) * a.G + (rem >> 3);
  return *slot < a.slots;
}
static unsigned place_blocks(const LinearArgs& a) { return (unsigned)(((int64_t)a.slots * a.H + 7) / 8 * 8 * a.G); }

// Decays of one chunk, from the 64 log decays in a wave's lanes. The sums are kept in 64 bits (as two 32-bit
// floats, in powers of two): differences of 32-bit sums of strong decays would lose what they differ by.
// A log decay under -10000 is taken as that: its exponential is 0 either way, and infinities have no differences.
struct Decays {
  float hi[CH], lo[CH]; // sum up to and with each token
  float in[CH];         // factor of the state that enters, for each row
  float w[CH];          // factor of each row in the state that leaves
  float all;            // factor of the state that enters in the one that leaves
};
__device__ __forceinline__ double up(double x, int by, int lane) {
  const double y = __shfl_up(x, by);
  return lane >= by ? x + y : x;
}
template <bool REV>
__device__ __forceinline__ void chunk_decays(Decays& d, float g, float in_scale, float w_scale) {
  const int lane = threadIdx.x & 63;
  double s = (double)(g < -1e4f ? -1e4f : g) * 1.4426950408889634;
#pragma unroll
  for (int by = 1; by < 64; by *= 2) s = up(s, by, lane);
  const double total = __shfl(s, 63);
  const float begun = __builtin_amdgcn_exp2f((float)s), left = __builtin_amdgcn_exp2f((float)(total - s));
  d.hi[lane] = (float)s;
  d.lo[lane] = (float)(s - (double)(float)s);
  d.in[lane] = in_scale * (REV ? left : begun);
  d.w[lane] = w_scale * (REV ? begun : left);
  if (lane == 63) d.all = begun;
}
__device__ __forceinline__ float log_decay(const LinearArgs& a, int h, int t, int t1) {
  return t < t1 ? a.g[(int64_t)t * a.gs + h] : 0.f;
}

// 64 rows of an operand: through a buffer that ends with the segment, so that rows behind it are zeros
template <typename T, int D>
struct Rows {
  static constexpr int PER = 16 / sizeof(T), PIECES = CH * D / PER / NTHREADS, STRIDE = D + Op<T>::PADDED;
  i32x4_t r[PIECES];
  __device__ __forceinline__ void load(const LinearSide& x, const LinearArgs& a, int h, int t, int t1) {
    const int n = max(min(t1 - t, CH), 0);
    const T* p = (const T*)x.p + (int64_t)t * x.stride + (int64_t)(x.shared ? h / a.G : h) * D;
    const __amdgpu_buffer_rsrc_t from = make_rsrc(p, n > 0 ? ((n - 1) * (int)x.stride + D) * (int)sizeof(T) : 0);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = threadIdx.x + i * NTHREADS, row = at / (D / PER), col = at % (D / PER) * PER;
      r[i] = buf_load16(from, row < n ? (row * (int)x.stride + col) * (int)sizeof(T) : 0x7ffffff0);
    }
  }
  __device__ __forceinline__ void store(T* tile) const {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = threadIdx.x + i * NTHREADS, row = at / (D / PER), col = at % (D / PER) * PER;
      *reinterpret_cast<i32x4_t*>(tile + row * STRIDE + col) = r[i];
    }
  }
};

// W += b^T diag(w) c over one chunk, for a wave's columns: W[kt][ct] the 16x16 tile of rows 16 kt.. and columns
// col0 + 16 ct... w c is the one operand that is no input; it goes in as EXACT terms, since the states are
// results in FP32 and everything after them is made from them.
template <typename T, int D, int CT>
__device__ __forceinline__ void add_to_state(f32x4 (&W)[D / 16][CT], const typename Op<T>::frag (&cf)[2][CT], const T* tb,
                                             const Decays& d) {
  constexpr int LD = Rows<T, D>::STRIDE, NT = Op<T>::EXACT;
  const int g = (threadIdx.x & 63) >> 4;
  const float all = d.all;
#pragma unroll
  for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) W[kt][ct] *= all;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    const f32x8 w = join(*reinterpret_cast<const f32x4*>(&d.w[32 * ks + 4 * g]), *reinterpret_cast<const f32x4*>(&d.w[32 * ks + 16 + 4 * g]));
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const Terms<T, NT> cw(widen<T>(cf[ks][ct]) * w);
#pragma unroll
      for (int kt = 0; kt < D / 16; ++kt) W[kt][ct] = mul_terms<T, NT>(Op<T>::down(tb, LD, 32 * ks, 16 * kt), cw, W[kt][ct]);
    }
  }
}

// ------------------------------------------------------------------------------------------------
// What each segment adds to a state, and its decay. The last segment of a document (the first, in reverse)
// is left out: no other starts from it.
template <typename T, int D, bool REV>
__global__ __launch_bounds__(NTHREADS, sizeof(T) == 2 ? 2 : 1) void k_linear_states(LinearArgs a) {
  constexpr int CT = D / 64, LD = Rows<T, D>::STRIDE;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  T* tb = (T*)lds;
  T* tc = tb + CH * LD;
  Decays* dec = (Decays*)(tc + CH * LD);
  int slot, h;
  if (!place(a, &slot, &h)) return;
  const Segment s = find_segment(a, slot);
  if (!s.live || (REV ? s.first : s.last)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15, col0 = wave * 16 * CT;
  f32x4 W[D / 16][CT];
#pragma unroll
  for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) W[kt][ct] = zero4();
  const int chunks = (s.t1 - s.t0 + CH - 1) / CH;
  const auto at = [&](int i) { return s.t0 + (REV ? chunks - 1 - i : i) * CH; };
  Rows<T, D> rb, rc;
  float gl = 0.f;
  double sum = 0.0; // of the log decays, in wave 0
  rb.load(a.b, a, h, at(0), s.t1);
  rc.load(a.c, a, h, at(0), s.t1);
  if (wave == 0) gl = log_decay(a, h, at(0) + lane, s.t1);
  for (int i = 0; i < chunks; ++i) {
    rb.store(tb);
    rc.store(tc);
    if (wave == 0) {
      chunk_decays<REV>(*dec, gl, 1.f, a.w_scale);
      sum += (double)(gl < -1e4f ? -1e4f : gl);
    }
    __syncthreads();
    if (i + 1 < chunks) {
      rb.load(a.b, a, h, at(i + 1), s.t1);
      rc.load(a.c, a, h, at(i + 1), s.t1);
      if (wave == 0) gl = log_decay(a, h, at(i + 1) + lane, s.t1);
    }
    typename Op<T>::frag cf[2][CT];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) cf[ks][ct] = Op<T>::down(tc, LD, 32 * ks, col0 + 16 * ct);
    add_to_state<T, D, CT>(W, cf, tb, *dec);
    __syncthreads();
  }
  float* to = a.states + ((int64_t)slot * a.HV + h) * D * D;
#pragma unroll
  for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int e = 0; e < 4; ++e) to[(16 * kt + 4 * g + e) * D + col0 + 16 * ct + l16] = W[kt][ct][e];
  if (wave == 0) {
#pragma unroll
    for (int by = 32; by > 0; by >>= 1) sum += __shfl_xor(sum, by);
    if (lane == 0) a.decay[(int64_t)slot * a.HV + h] = __builtin_amdgcn_exp2f((float)(sum * 1.4426950408889634));
  }
}

// The states that segments start from, in place of what they add: forward from `init` (h0) at the first segment,
// reverse from `init` (dht) at the last.
template <bool REV>
__global__ __launch_bounds__(256) void k_linear_scan(LinearArgs a) {
  const int n = blockIdx.z, h = blockIdx.y, size = a.D * a.D;
  const int e = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= size) return;
  const int from = cut_to(a.cu[n], a.T), to = max(cut_to(a.cu[n + 1], a.T), from);
  const int count = (to - from + a.seg - 1) / a.seg, base = doc_slot(a, n);
  const auto slot = [&](int i) { return base + (REV ? count - 1 - i : i); };
  const auto at = [&](int i) { return a.states + ((int64_t)slot(i) * a.HV + h) * size + e; };
  f32x4 W = zero4();
  if (a.init) W = *reinterpret_cast<const f32x4*>(a.init + ((int64_t)n * a.HV + h) * size + e);
  constexpr int AHEAD = 4;
  for (int i = 0; i < count; i += AHEAD) {
    f32x4 add[AHEAD];
    float dec[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      add[j] = zero4();
      dec[j] = 0.f;
      if (i + j < count - 1) {
        add[j] = *reinterpret_cast<const f32x4*>(at(i + j));
        dec[j] = a.decay[(int64_t)slot(i + j) * a.HV + h];
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (i + j < count && i + j > 0) *reinterpret_cast<f32x4*>(at(i + j)) = W;
      W = W * dec[j] + add[j];
    }
  }
}

// ------------------------------------------------------------------------------------------------
// The walk. A wave owns 16 CT columns of the state W (and of c and y) and keeps them in registers for the
// whole segment; a chunk takes
//   y^T  = W^T a^T, each column times its row's factor       (W's registers are the operand as they are)
//   P    = decays * a b^T, its 16x16 tiles shared out to the waves, through LDS
//   y^T += c^T P^T                                            (written out: 4 neighbouring columns a lane)
//   W    = decay W + b^T diag(w) c
// P and W's operand are rounded once, to the io type: their products are summed in FP32 and the result is
// rounded to that type itself. With `dots` (the decays' gradient, an FP32 result that is a difference of
// sums) both go in as EXACT terms instead.
template <typename T, int D, bool REV, bool DOTS>
__global__ __launch_bounds__(NTHREADS, sizeof(T) == 2 ? 2 : 1) void k_linear_walk(LinearArgs a) {
  constexpr int CT = D / 64, LD = Rows<T, D>::STRIDE, NT = DOTS ? Op<T>::EXACT : 1;
  typedef typename std::conditional<DOTS, float, T>::type PT; // type of P in LDS
  constexpr int LP = CH + Op<PT>::PADDED;
  typedef typename Op<T>::frag frag;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  T* ta = (T*)lds;
  T* tb = ta + CH * LD;
  T* tc = tb + CH * LD;
  PT* tp = (PT*)(tc + CH * LD);
  Decays* dec = (Decays*)(tp + CH * LP);
  float* red = (float*)(dec + 1); // DOTS: [4 waves][64 rows]
  int slot, h;
  if (!place(a, &slot, &h)) return;
  const Segment s = find_segment(a, slot);
  if (!s.live) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int col0 = wave * 16 * CT;
  const int64_t doc_state = ((int64_t)s.doc * a.HV + h) * D * D;

  // the state: rows 16 kt + 4 g + e, column col0 + 16 ct + l16; `flip`: stored with rows and columns exchanged
  f32x4 W[D / 16][CT];
  const bool begins = REV ? s.last : s.first;
  const float* from = begins ? (a.init ? a.init + doc_state : nullptr) : a.states + ((int64_t)slot * a.HV + h) * D * D;
#pragma unroll
  for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int row = 16 * kt + 4 * g, col = col0 + 16 * ct + l16;
      W[kt][ct] = zero4();
      if (from) {
        if (a.flip) W[kt][ct] = *reinterpret_cast<const f32x4*>(from + col * D + row);
        else
#pragma unroll
          for (int e = 0; e < 4; ++e) W[kt][ct][e] = from[(row + e) * D + col];
      }
    }

  // the tiles of P beside the diagonal that products read but no wave writes
  for (int i = threadIdx.x; i < CH * CH; i += NTHREADS) tp[(i / CH) * LP + i % CH] = (PT)0.f;

  const int chunks = (s.t1 - s.t0 + CH - 1) / CH;
  const auto at = [&](int i) { return s.t0 + (REV ? chunks - 1 - i : i) * CH; };
  Rows<T, D> ra, rb, rc;
  float gl = 0.f;
  if (chunks > 0) {
    ra.load(a.a, a, h, at(0), s.t1);
    rb.load(a.b, a, h, at(0), s.t1);
    rc.load(a.c, a, h, at(0), s.t1);
    if (wave == 3) gl = log_decay(a, h, at(0) + lane, s.t1);
  }
  for (int i = 0; i < chunks; ++i) {
    const int t = at(i), n = min(s.t1 - t, CH);
    Decays& d = *dec;
    ra.store(ta);
    rb.store(tb);
    rc.store(tc);
    if (wave == 3) chunk_decays<REV>(d, gl, a.in_scale, a.w_scale);
    __syncthreads();
    if (i + 1 < chunks) {
      ra.load(a.a, a, h, at(i + 1), s.t1);
      rb.load(a.b, a, h, at(i + 1), s.t1);
      rc.load(a.c, a, h, at(i + 1), s.t1);
      if (wave == 3) gl = log_decay(a, h, at(i + 1) + lane, s.t1);
    }
    // P^T: rows s, column t; tiles (tb, sb) with sb <= tb, (sb, tb) exchanged in reverse
#pragma unroll 1
    for (int e = wave; e < 10; e += 4) {
      const int x = e < 1 ? 0 : e < 3 ? 1 : e < 6 ? 2 : 3, y = e - x * (x + 1) / 2;
      const int bt = REV ? y : x, bs = REV ? x : y;
      f32x4 p = zero4();
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk)
        p = Op<T>::mul(Op<T>::along(tb, LD, 16 * bs + l16, 32 * kk), Op<T>::along(ta, LD, 16 * bt + l16, 32 * kk), p);
      const int tt = 16 * bt + l16, ss = 16 * bs + 4 * g;
      const float th = d.hi[tt], tl = d.lo[tt];
      const f32x4 sh = *reinterpret_cast<const f32x4*>(&d.hi[ss]), sl = *reinterpret_cast<const f32x4*>(&d.lo[ss]);
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x2 = REV ? (sh[j] - th) + (sl[j] - tl) : (th - sh[j]) + (tl - sl[j]);
        const bool keep = REV ? ss + j >= tt : ss + j <= tt;
        v[j] = keep ? a.p_scale * p[j] * __builtin_amdgcn_exp2f(x2) : 0.f;
      }
      IO<PT>::store4(tp + tt * LP + ss, v);
    }
    // y^T = W^T a^T
    f32x4 y[CT][4];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int bt = 0; bt < 4; ++bt) y[ct][bt] = zero4();
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
      frag af[4];
#pragma unroll
      for (int bt = 0; bt < 4; ++bt) af[bt] = Op<T>::along(ta, LD, 16 * bt + l16, 32 * kk);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const Terms<T, NT> w(join(W[2 * kk][ct], W[2 * kk + 1][ct]));
#pragma unroll
        for (int bt = 0; bt < 4; ++bt) y[ct][bt] = mul_terms<T, NT>(w, af[bt], y[ct][bt]);
      }
    }
#pragma unroll
    for (int bt = 0; bt < 4; ++bt) {
      const float f = d.in[16 * bt + l16];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) y[ct][bt] *= f;
    }
    frag cf[2][CT];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) cf[ks][ct] = Op<T>::down(tc, LD, 32 * ks, col0 + 16 * ct);
    __syncthreads(); // P
#pragma unroll
    for (int bt = 0; bt < 4; ++bt)
#pragma unroll
      for (int ks = REV ? bt / 2 : 0; ks < (REV ? 2 : bt / 2 + 1); ++ks) {
        if constexpr (DOTS) {
          const float* p = (const float*)tp + (16 * bt + l16) * LP + 32 * ks + 4 * g;
          const Terms<T, NT> pf(join(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 16)));
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) y[ct][bt] = mul_terms<T, NT>(cf[ks][ct], pf, y[ct][bt]);
        } else {
          const frag pf = Op<T>::along((const T*)tp, LP, 16 * bt + l16, 32 * ks);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) y[ct][bt] = Op<T>::mul(cf[ks][ct], pf, y[ct][bt]);
        }
      }
    add_to_state<T, D, CT>(W, cf, tb, d);

    // y: lane (g, l16): row 16 bt + l16, columns col0 + 16 ct + 4 g .. + 3
    const auto write = [&](auto* out) {
      typedef typename std::remove_reference<decltype(*out)>::type O;
      const int os = a.HV * D;
      const __amdgpu_buffer_rsrc_t to = make_rsrc(out + (int64_t)t * os + (int64_t)h * D, ((n - 1) * os + D) * (int)sizeof(O));
#pragma unroll
      for (int bt = 0; bt < 4; ++bt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const int row = 16 * bt + l16;
          const float v[4] = {y[ct][bt][0], y[ct][bt][1], y[ct][bt][2], y[ct][bt][3]};
          if (row < n) IO<O>::bstore4(to, row * os + col0 + 16 * ct + 4 * g, v);
        }
    };
    if (a.part) write(a.part);
    else write((T*)a.out);
    if constexpr (DOTS) {
#pragma unroll
      for (int bt = 0; bt < 4; ++bt) {
        const int row = 16 * bt + l16;
        const T* x = (const T*)a.dot.p + (int64_t)(t + min(row, n - 1)) * a.dot.stride + (int64_t)(a.dot.shared ? h / a.G : h) * D + col0 + 4 * g;
        float sum = 0.f;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum = __builtin_fmaf((float)x[16 * ct + e], y[ct][bt][e], sum);
        sum = col_sum4(sum);
        if (g == 0) red[wave * CH + row] = sum;
      }
    }
    __syncthreads();
    if constexpr (DOTS) {
      if ((int)threadIdx.x < n)
        a.dots[(int64_t)h * a.T + t + threadIdx.x] =
            (red[threadIdx.x] + red[CH + threadIdx.x]) + (red[2 * CH + threadIdx.x] + red[3 * CH + threadIdx.x]);
    }
  }
  if ((REV ? s.first : s.last) && a.fin) {
    float* to = a.fin + doc_state;
#pragma unroll
    for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int e = 0; e < 4; ++e) to[(16 * kt + 4 * g + e) * D + col0 + 16 * ct + l16] = W[kt][ct][e];
  }
}

// ------------------------------------------------------------------------------------------------
// Sum over the value heads of a group, in their order: part f32 [T, HV, D] -> out [T, H, D]
template <typename T>
__global__ __launch_bounds__(256) void k_linear_group_sum(LinearArgs a) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, n = (int64_t)a.T * a.H * a.D;
  if (i >= n) return;
  const int64_t head = i / a.D, col = i - head * a.D;
  const float* p = a.part + head * a.G * a.D + col;
  f32x4 s = *reinterpret_cast<const f32x4*>(p);
  for (int j = 1; j < a.G; ++j) s += *reinterpret_cast<const f32x4*>(p + (int64_t)j * a.D);
  const float v[4] = {s[0], s[1], s[2], s[3]};
  IO<T>::store4((T*)a.out + i, v);
}

// ------------------------------------------------------------------------------------------------
// The decays' gradient. Summed over a whole document the differences q.dq - k.dk would lose what is left of
// them, so each segment starts again from its border, where the gradient is <S, D> of the state there and its
// own gradient, both at hand: dg_t = <S_end, D_end> + sum_{s >= t} (q_s.dq_s - k_s.dk_s). A document's last segment has no
// S_end: without dht its D_end is 0; with it the sum runs from the segment's start instead, where S_0 = 0 or
// both S_0 and D_0 are at hand: dg_t = <S_0, D_0> - sum_{s < t} (q_s.dq_s - k_s.dk_s).
__device__ __forceinline__ double block_sum(double x, double* tmp) {
#pragma unroll
  for (int by = 32; by > 0; by >>= 1) x += __shfl_xor(x, by);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
  __syncthreads();
  return (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
}
__global__ __launch_bounds__(256) void k_linear_dg(LinearDgArgs d) {
  const LinearArgs& a = d.a;
  __shared__ double tmp[4], carry[4];
  const int slot = blockIdx.x, h = blockIdx.y, size = a.D * a.D;
  const Segment s = find_segment(a, slot);
  const auto state = [&](const float* base, int64_t at) { return base + (at * a.HV + h) * size; };
  const float *x = nullptr, *y = nullptr; // S and D at the border
  bool from_end = true;
  if (s.live) {
    if (!s.last) {
      x = state(d.S, slot + 1);
      y = state(d.D, slot);
    } else if (d.dht) {
      from_end = false;
      if (s.i > 0) {
        x = state(d.S, slot);
        y = state(d.D, slot - 1);
      } else if (d.h0) {
        x = state(d.h0, s.doc);
        y = state(d.dh0, s.doc);
      }
    }
  }
  double f = 0.0;
  if (x)
    for (int e = threadIdx.x * 4; e < size; e += 1024) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(x + e), v = *reinterpret_cast<const f32x4*>(y + e);
      f += ((double)u[0] * v[0] + (double)u[1] * v[1]) + ((double)u[2] * v[2] + (double)u[3] * v[3]);
    }
  f = block_sum(f, tmp);
  double all = 0.0; // one decay a head: the sum of dg over the segment
  const int n = s.live ? s.t1 - s.t0 : 0;
  const float *qd = d.qdots + (int64_t)h * a.T + s.t0, *kd = d.kdots + (int64_t)h * a.T + s.t0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int c = 0; c < n; c += 256) { // from the border inwards
    const int j = c + (int)threadIdx.x, t = from_end ? n - 1 - j : j;
    const double own = j < n ? (double)qd[t] - (double)kd[t] : 0.0;
    double p = own;
#pragma unroll
    for (int by = 1; by < 64; by *= 2) p = up(p, by, lane);
    if (lane == 63) carry[wave] = p;
    __syncthreads();
    double before = 0.0, turn = 0.0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      before += w < wave ? carry[w] : 0.0;
      turn += carry[w];
    }
    const double v = from_end ? f + before + p : f - before - (p - own);
    if (j < n) {
      if (a.gs) d.dg[(int64_t)(s.t0 + t) * a.HV + h] = (float)v;
      all += v;
    }
    f += from_end ? turn : -turn;
    __syncthreads();
  }
  if (a.gs == 0) {
    all = block_sum(all, tmp);
    if (threadIdx.x == 0) d.sums[(int64_t)slot * a.HV + h] = all;
  }
}
// One decay a head: the segments' sums, in their order.
__global__ __launch_bounds__(256) void k_linear_dg_sum(LinearDgArgs d) {
  __shared__ double tmp[4];
  const int h = blockIdx.x;
  double s = 0.0;
  for (int i = threadIdx.x; i < d.a.slots; i += 256) s += d.sums[(int64_t)i * d.a.HV + h];
  s = block_sum(s, tmp);
  if (threadIdx.x == 0) d.dg[h] = (float)s;
}

// ------------------------------------------------------------------------------------------------
// More LDS than the runtime gives unasked is asked for once on each device.
static int ask_lds(const void* kernel, unsigned lds, std::atomic<uint64_t>& asked) {
  if (lds <= 64 * 1024) return 0;
  int dev = 0;
  if (const hipError_t e = hipGetDevice(&dev)) return (int)e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (asked.load(std::memory_order_relaxed) & bit) return 0;
  const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return (int)e;
  asked.fetch_or(bit, std::memory_order_relaxed);
  return 0;
}

template <typename T, int D, bool REV>
static int states_t(const LinearArgs& a, hipStream_t s) {
  constexpr unsigned lds = 2 * CH * Rows<T, D>::STRIDE * sizeof(T) + sizeof(Decays);
  static std::atomic<uint64_t> asked{0};
  if (const int e = ask_lds(reinterpret_cast<const void*>(&k_linear_states<T, D, REV>), lds, asked)) return e;
  hipLaunchKernelGGL((k_linear_states<T, D, REV>), dim3(place_blocks(a)), dim3(NTHREADS), lds, s, a);
  return (int)hipGetLastError();
}
template <typename T, int D>
static int states_td(const LinearArgs& a, bool rev, hipStream_t s) {
  return rev ? states_t<T, D, true>(a, s) : states_t<T, D, false>(a, s);
}
template <typename T, int D, bool REV, bool DOTS>
static int walk_t(const LinearArgs& a, hipStream_t s) {
  constexpr unsigned lds = 3 * CH * Rows<T, D>::STRIDE * sizeof(T) +
                           (DOTS ? CH * (CH + Op<float>::PADDED) * 4 : CH * (CH + Op<T>::PADDED) * (unsigned)sizeof(T)) +
                           sizeof(Decays) + (DOTS ? 4 * CH * 4 : 0);
  static std::atomic<uint64_t> asked{0};
  if (const int e = ask_lds(reinterpret_cast<const void*>(&k_linear_walk<T, D, REV, DOTS>), lds, asked)) return e;
  hipLaunchKernelGGL((k_linear_walk<T, D, REV, DOTS>), dim3(place_blocks(a)), dim3(NTHREADS), lds, s, a);
  return (int)hipGetLastError();
}
template <typename T, int D>
static int walk_td(const LinearArgs& a, bool rev, hipStream_t s) {
  if (rev) return a.dots ? walk_t<T, D, true, true>(a, s) : walk_t<T, D, true, false>(a, s);
  return a.dots ? walk_t<T, D, false, true>(a, s) : walk_t<T, D, false, false>(a, s);
}

int launch_linear_states(const LinearArgs& a, bool rev, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == 0) return a.D == 128 ? states_td<bf16, 128>(a, rev, s) : states_td<bf16, 64>(a, rev, s);
  return a.D == 128 ? states_td<float, 128>(a, rev, s) : states_td<float, 64>(a, rev, s);
}

int launch_linear_scan(const LinearArgs& a, bool rev, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)((a.D * a.D + 1023) / 1024), (unsigned)a.HV, (unsigned)a.N);
  if (rev) hipLaunchKernelGGL(k_linear_scan<true>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_linear_scan<false>, grid, dim3(256), 0, s, a);
  return (int)hipGetLastError();
}

int launch_linear_walk(const LinearArgs& a, bool rev, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == 0) return a.D == 128 ? walk_td<bf16, 128>(a, rev, s) : walk_td<bf16, 64>(a, rev, s);
  return a.D == 128 ? walk_td<float, 128>(a, rev, s) : walk_td<float, 64>(a, rev, s);
}

int launch_linear_group_sum(const LinearArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int64_t n = (int64_t)a.T * a.H * a.D / 4;
  const dim3 grid((unsigned)((n + 255) / 256));
  if (dtype == 0) hipLaunchKernelGGL(k_linear_group_sum<bf16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_linear_group_sum<float>, grid, dim3(256), 0, s, a);
  return (int)hipGetLastError();
}

int launch_linear_dg(const LinearDgArgs& d, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(k_linear_dg, dim3((unsigned)d.a.slots, (unsigned)d.a.HV), dim3(256), 0, s, d);
  if (const int e = (int)hipGetLastError()) return e;
  if (d.a.gs) return 0;
  hipLaunchKernelGGL(k_linear_dg_sum, dim3((unsigned)d.a.HV), dim3(256), 0, s, d);
  return (int)hipGetLastError();
}

} // namespace gdn
