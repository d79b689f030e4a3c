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

// ------------------------------------------------------------------------------------------------
// Tiles: 64 rows of d values in LDS, filled straight from memory (16 bytes a lane, a wave's lanes next to each
// other), so rows are not padded. Instead the 16-byte unit u of row r lies at u ^ f(r mod 16), where f is chosen
// so that the lanes that are served together meet all 64 banks, both where they read along rows (16 rows,
// 8 bytes each for bf16, 16 for f32) and down columns (bf16: 8 rows, 32 bytes each; f32: 4 rows, 64 bytes each).
//
// Operands of 16x16 products over 32 k values come in the k-permuted order of gdn_device.h: lane group g has the
// k values 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3. bf16 rows go to one instruction, f32 rows to eight of
// 4 k values (element e of every lane to the e-th), so both share all of the indexing.
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;

template <typename T>
__device__ __forceinline__ T lds_read(int at) {
  return *(__attribute__((address_space(3))) const T*)(lds_char*)(uintptr_t)at;
}
template <typename T>
__device__ __forceinline__ void lds_write(int at, const T& x) {
  *(__attribute__((address_space(3))) T*)(lds_char*)(uintptr_t)at = x;
}

template <typename T, int D>
struct Tile {
  static constexpr bool HALF = sizeof(T) == 2;
  static constexpr int ROW = D * sizeof(T), BYTES = CH * ROW; // of a row, of a tile
  static constexpr int UNITS = ROW / 16, TOGETHER = 64 / UNITS, PIECES = 16 / TOGETHER; // rows a load, loads of a wave's 16 rows
  static __device__ __forceinline__ constexpr int f(int r) {
    return !HALF ? r & 15 : D == 128 ? (r & 7) << 1 | (r >> 3 & 1) : (r >> 1 & 3) << 1 | (r >> 3 & 1);
  }
};

template <typename T>
struct Op;
template <>
struct Op<bf16> {
  typedef bf16x8 frag;
  // The terms that hold an FP32 value: 3 bf16 hold all of its 24 bits.
  static constexpr int EXACT = 3;
  // lane constants: of a read along row l16 (of 16), down the column of lane l16 (of 16) from row 4 g
  template <int D>
  static __device__ __forceinline__ int along_lane() {
    typedef Tile<bf16, D> S;
    const int l = threadIdx.x & 63, g = l >> 4, r = l & 15;
    return r * S::ROW + (((g >> 1) ^ S::f(r)) << 4) + (g & 1) * 8;
  }
  template <int D> // rows 16 row16 .., k values 32 kk ..
  static __device__ __forceinline__ frag along(int tile, int lane, int row16, int kk) {
    const int at = tile + row16 * 16 * Tile<bf16, D>::ROW;
    const bf16x4 a = lds_read<bf16x4>(at + (lane ^ (kk << 6))), b = lds_read<bf16x4>(at + (lane ^ (kk << 6 | 32)));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  // Columns `first` + `step` (l16 / 4) + l16 mod 4, both multiples of 4. The transposing read hands lane i of 16 element
  // i mod 4 of the 8-byte blocks that lanes i / 4, + 4, .. address (see lds_tr8).
  struct Down {
    int at;
  };
  template <int D>
  static __device__ __forceinline__ Down down_lane(int first, int step) {
    typedef Tile<bf16, D> S;
    const int l = threadIdx.x & 63, g = l >> 4, j = l & 15, r = 4 * g + (j >> 2), col = first + step * (j & 3);
    return {r * S::ROW + (((col >> 3) ^ S::f(r)) << 4) + (col & 4) * 2};
  }
  template <int D> // k values: rows 32 ks ..; columns moved by 16 m
  static __device__ __forceinline__ frag down(int tile, const Down& lane, int ks, int m) {
    constexpr int ROW = Tile<bf16, D>::ROW;
    typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
    const int at = ((tile + lane.at) ^ (m << 5)) + 32 * ks * ROW; // (a tile's address has none of the bits exchanged)
    const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(lds_char*)(uintptr_t)at);
    const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(lds_char*)(uintptr_t)(at + 16 * ROW));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ f32x4 mul(const frag& a, const frag& b, const f32x4& c) { return mfma(a, b, c); }
};
template <>
struct Op<float> {
  typedef f32x8 frag;
  static constexpr int EXACT = 1;
  template <int D>
  static __device__ __forceinline__ int along_lane() {
    typedef Tile<float, D> S;
    const int l = threadIdx.x & 63, g = l >> 4, r = l & 15;
    return r * S::ROW + ((g ^ S::f(r)) << 4);
  }
  template <int D>
  static __device__ __forceinline__ frag along(int tile, int lane, int row16, int kk) {
    const int at = tile + row16 * 16 * Tile<float, D>::ROW;
    const f32x4 a = lds_read<f32x4>(at + (lane ^ (kk << 7))), b = lds_read<f32x4>(at + (lane ^ (kk << 7 | 64)));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  struct Down {
    int at[4];
  };
  template <int D>
  static __device__ __forceinline__ Down down_lane(int first, int step) {
    typedef Tile<float, D> S;
    const int l = threadIdx.x & 63, g = l >> 4, j = l & 15, col = first + step * (j >> 2);
    Down d;
#pragma unroll
    for (int e = 0; e < 4; ++e) d.at[e] = (4 * g + e) * S::ROW + (((col >> 2) ^ S::f(4 * g + e)) << 4) + (j & 3) * 4;
    return d;
  }
  template <int D>
  static __device__ __forceinline__ frag down(int tile, const Down& lane, int ks, int m) {
    constexpr int ROW = Tile<float, D>::ROW;
    frag r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = ((tile + lane.at[e]) ^ (m << 6)) + 32 * ks * ROW;
      r[e] = lds_read<float>(at);
      r[4 + e] = lds_read<float>(at + 16 * ROW);
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
// before it left (x - x's leading bits by a product with -1: exact, and one instruction from the packed pair).
template <typename T, int NT>
struct Terms {
  typename Op<T>::frag f[NT];
  __device__ __forceinline__ Terms() {}
  __device__ __forceinline__ explicit Terms(const f32x8& x) {
    if constexpr (sizeof(T) == 4) {
      f[0] = x;
    } else {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      // (-1, 0) and (0, -1); as a constant that the compiler knows it would become an inline one, which the
      // instruction reads as a 32-bit -1
      unsigned low = 0xbf80, high = 0xbf800000;
      asm("" : "+s"(low), "+s"(high));
      const bf16x2 first = __builtin_bit_cast(bf16x2, low), second = __builtin_bit_cast(bf16x2, high);
      f32x8 left = x;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const bf16x2 h = {(__bf16)left[e], (__bf16)left[e + 1]};
          f[n][e] = h[0];
          f[n][e + 1] = h[1];
          if (n + 1 < NT) {
            left[e] = __builtin_amdgcn_fdot2_f32_bf16(h, first, left[e], false);
            left[e + 1] = __builtin_amdgcn_fdot2_f32_bf16(h, second, left[e + 1], false);
          }
        }
    }
  }
};
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
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int cut_to(int x, int T) { return min(max(x, 0), T); }
__device__ __forceinline__ int doc_slot(const LinearArgs& a, int n) { return a.seg == 0 ? n : cut_to(a.cu[n], a.T) / a.seg + n; }
__device__ __forceinline__ Segment find_segment(const LinearArgs& a, int slot) {
  int lo = 0, hi = a.N - 1; // the last document whose first slot is at most `slot`
  if (a.seg == 0) lo = slot;
  else
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (uniform(doc_slot(a, mid)) <= slot) lo = mid;
      else hi = mid - 1;
    }
  Segment s;
  s.doc = lo;
  const int from = uniform(cut_to(a.cu[lo], a.T)), to = max(uniform(cut_to(a.cu[lo + 1], a.T)), from);
  s.i = a.seg == 0 ? 0 : slot - uniform(doc_slot(a, lo));
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
__device__ __forceinline__ bool place(const LinearArgs& a, int b, int* slot, int* h) {
  const int per = 8 * a.G;
  const int sg = b / per, rem = b - sg * per;
  const int group = sg * 8 + (rem & 7);
  *slot = group / a.H;
  *h = (group - *slot * a.H) * a.G + (rem >> 3);
  return *slot < a.slots;
}
// Launches of many workgroups have two dimensions: one holds less than 2^32 threads.
constexpr unsigned MOST_BLOCKS = 1 << 20;
__device__ __forceinline__ int block_index() { return (int)(blockIdx.y * gridDim.x + blockIdx.x); }
static dim3 many_blocks(unsigned n) { return n <= MOST_BLOCKS ? dim3(n) : dim3(MOST_BLOCKS, (n + MOST_BLOCKS - 1) / MOST_BLOCKS); }
static unsigned place_blocks(const LinearArgs& a) { return (unsigned)(((int64_t)a.slots * a.H + 7) / 8 * 8 * a.G); }

// Decays of one chunk, from the 64 log decays in a wave's lanes. The sums are kept in 64 bits (as two 32-bit
// floats, in powers of two): differences of 32-bit sums of strong decays would lose what they differ by.
// A log decay under -10000 is taken as that: its exponential is 0 either way, and infinities have no differences.
struct alignas(16) Decays {
  float hi[CH], lo[CH]; // sum up to and with each token
  float in[CH];         // factor of the state that enters, for each row
  float w[CH];          // factor of each row in the state that leaves
  float all;            // factor of the state that enters in the one that leaves
};
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double x) { // lanes without a source add 0
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)b, CTRL, ROWS, 0xf, false);
  const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), CTRL, ROWS, 0xf, false);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Inclusive sums over a wave's lanes, by the steps of wave_prefix_sum.
__device__ __forceinline__ double wave_sums(double x) {
  x = scan_step<0x111, 0xf>(x);
  x = scan_step<0x112, 0xf>(x);
  x = scan_step<0x114, 0xf>(x);
  x = scan_step<0x118, 0xf>(x);
  x = scan_step<0x142, 0xa>(x);
  return scan_step<0x143, 0xc>(x);
}
__device__ __forceinline__ double last_lane(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)b, 63), hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(b >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <bool REV>
__device__ __forceinline__ void chunk_decays(Decays& d, float g, float in_scale, float w_scale) {
  const int lane = threadIdx.x & 63;
  const double s = wave_sums((double)(g < -1e4f ? -1e4f : g) * 1.4426950408889634), total = last_lane(s);
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

// 64 rows of an operand from memory to a tile: wave w loads rows 16 w .. of it, through a buffer that ends with
// the segment, so that rows behind it arrive as zeros. The loads are written in assembly, without output
// registers: the compiler, which cannot tell one tile from another, would wait for them before every read of any
// tile. They are waited for by wait_loads before the barrier that hands the tile over. m0 (where in LDS a wave's lanes write) is
// an operand, so that the compiler sets it and knows until when it is needed; the s_nop stands between the two.
template <typename T, int D>
struct Feed {
  typedef Tile<T, D> S;
  const T* base; // of the head
  int stride, unit, lane, wave; // the lane's place in a row and its row, in bytes
  __device__ __forceinline__ Feed(const LinearSide& x, const LinearArgs& a, int h, int w)
      : base((const T*)x.p + (int64_t)(x.shared ? h / a.G : h) * D), stride((int)x.stride), wave(w) {
    const int l = threadIdx.x & 63, q = l / S::UNITS, u = l % S::UNITS;
    unit = (u ^ S::f(q)) << 4;
    lane = q * stride * (int)sizeof(T);
  }
  __device__ __forceinline__ void load(int tile, int t, int t1) const {
    const int n = max(min(t1 - t, CH), 0);
    const uint64_t p = (uint64_t)(base + (int64_t)t * stride);
    i32x4_t from = {uniform((int)p), uniform((int)(p >> 32) & 0xffff), uniform(n > 0 ? ((n - 1) * stride + D) * (int)sizeof(T) : 0),
                    0x00020000}; // make_rsrc's words
    asm volatile("s_nop 4" : "+s"(from)); // before a buffer access reads scalars that a vector instruction wrote
    const int step = S::TOGETHER * stride * (int)sizeof(T);
    int row = wave * S::PIECES * step, to = uniform(tile + wave * 16 * S::ROW);
#pragma unroll
    for (int i = 0; i < S::PIECES; ++i, row += step, to += 1024) {
      const int off = (unit ^ (S::f(i * S::TOGETHER) << 4)) + lane + row;
      asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "{m0}"(to), "v"(off), "s"(from) : "memory");
    }
  }
};
// Waits until all but the newest N of a wave's memory accesses are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Column of lane l16 in a wave's tile ct of CT: neighbouring tiles share 4 CT neighbouring columns, so that a lane's
// part of a row of y is one piece.
template <int CT>
__device__ __forceinline__ int column(int col0, int ct, int l16) {
  return col0 + 4 * CT * (l16 >> 2) + 4 * ct + (l16 & 3);
}

// A value that the compiler takes for a new one: what is derived from it is computed where it is used, and not
// kept in registers from before a loop.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The states between the kernels lie as the registers hold them: four rows of a column together, a wave's lanes next to
// each other. Element i of that order is row kept_row(i), column kept_col(i).
template <int D>
__device__ __forceinline__ int kept_at(int wave, int kt, int ct, int lane) {
  return (((wave * (D / 16) + kt) * (D / 64) + ct) * 64 + lane) * 4;
}
template <int D>
__device__ __forceinline__ int kept_row(int i) {
  return 16 * (i / 256 / (D / 64) % (D / 16)) + 4 * (i / 64 % 4) + i % 4;
}
template <int D>
__device__ __forceinline__ int kept_col(int i) {
  return column<D / 64>(i / 256 / (D / 64) / (D / 16) * (D / 4), i / 256 % (D / 64), i / 4 % 16);
}
// And where the element of a row and column lies.
template <int D>
__device__ __forceinline__ int kept_of(int row, int col) {
  constexpr int CT = D / 64;
  const int in = col % (16 * CT), l16 = in / (4 * CT) * 4 + in % 4;
  return kept_at<D>(col / (16 * CT), row / 16, in / 4 % CT, row % 16 / 4 * 16 + l16) + row % 4;
}

// W = decay W + b^T diag(w) c over one chunk, for a wave's columns: W[kt][ct] the tile of rows 16 kt .. and the
// columns of tile ct, cf its c. w c is the one operand that is no input; it goes in as NT terms. (A tile's terms one
// after the other would wait for each other: a round over the tiles for each.)
template <typename T, int D, int CT, int NT>
__device__ __forceinline__ void add_to_state(f32x4 (&W)[D / 16][CT], const typename Op<T>::frag (&cf)[2][CT], int tb,
                                             const typename Op<T>::Down& lane, const Decays& d) {
  const int g = (threadIdx.x & 63) >> 4;
  const float all = d.all;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    const f32x8 w = join(*reinterpret_cast<const f32x4*>(&d.w[32 * ks + 4 * g]), *reinterpret_cast<const f32x4*>(&d.w[32 * ks + 16 + 4 * g]));
    Terms<T, NT> cw[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) cw[ct] = Terms<T, NT>(widen<T>(cf[ks][ct]) * w);
#pragma unroll
    for (int k4 = 0; k4 < D / 16; k4 += 4) {
      typename Op<T>::frag bf[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf[j] = Op<T>::template down<D>(tb, lane, ks, k4 + j);
        if (ks == 0)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) W[k4 + j][ct] *= all;
      }
#pragma unroll
      for (int n = NT - 1; n >= 0; --n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) W[k4 + j][ct] = Op<T>::mul(bf[j], cw[ct].f[n], W[k4 + j][ct]);
    }
  }
}

// LDS of the kernels: tiles at the start, then what they name. They have no other, so that it starts at address 0, and
// what lies at a fixed place in it is an offset in the instructions.
extern __shared__ __attribute__((aligned(1024))) char linear_lds[];

// ------------------------------------------------------------------------------------------------
// What each segment adds to a state, and its decay. The last segment of a document (the first, in reverse)
// is left out: no other starts from it. w c goes in as EXACT terms: the states are results in FP32, and
// everything after them is made from them. Bound by its matrix instructions and by the splitting between them: both
// directions of 32,768 tokens, 48 heads, 128 wide, 271 GFLOP in 290 us. Two workgroups a CU: one alone leaves it
// idle at its barriers (a chunk then takes 1.6 us, two of them 3.0).
template <typename T, int D, bool REV>
__device__ __forceinline__ void segment_state(const LinearArgs& a, int block) {
  typedef Tile<T, D> S;
  constexpr int CT = D / 64, NT = Op<T>::EXACT;
  Decays* dec = (Decays*)(linear_lds + 4 * S::BYTES); // of two chunks
  int slot, h;
  if (!place(a, block, &slot, &h)) return;
  const Segment s = find_segment(a, slot);
  if (!s.live || (REV ? s.first : s.last)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int col0 = wave * 16 * CT;
  f32x4 W[D / 16][CT];
#pragma unroll
  for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) W[kt][ct] = zero4();
  const int chunks = (s.t1 - s.t0 + CH - 1) / CH;
  const auto at = [&](int i) { return s.t0 + (REV ? chunks - 1 - i : i) * CH; };
  const Feed<T, D> fb(a.b, a, h, wave), fc(a.c, a, h, wave);
  const typename Op<T>::Down b_lane = Op<T>::template down_lane<D>(0, 4);
  typename Op<T>::Down c_lane[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) c_lane[ct] = Op<T>::template down_lane<D>(col0 + 4 * ct, 4 * CT);
  float gl = 0.f;
  double sum = 0.0; // of the log decays, in wave 0
  const auto decays = [&](int i) { // of chunk i, and the log decays of the next
    chunk_decays<REV>(dec[i & 1], gl, 1.f, a.w_scale);
    sum += (double)(gl < -1e4f ? -1e4f : gl);
    gl = i + 1 < chunks ? log_decay(a, h, at(i + 1) + lane, s.t1) : 0.f;
  };
  if (wave == 0) {
    gl = log_decay(a, h, at(0) + lane, s.t1);
    decays(0);
  }
  fb.load(0, at(0), s.t1);
  fc.load(S::BYTES, at(0), s.t1);
  const auto step = [&](int i, auto half) { // in tiles 2 half, 2 half + 1
    constexpr int tb = half * 2 * S::BYTES, tc = tb + S::BYTES, next = (1 - half) * 2 * S::BYTES;
    wait_loads<0>();
    __syncthreads();
    if (i + 1 < chunks) {
      fb.load(next, at(i + 1), s.t1);
      fc.load(next + S::BYTES, at(i + 1), s.t1);
    }
    typename Op<T>::frag cf[2][CT];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) cf[ks][ct] = Op<T>::template down<D>(tc, c_lane[ct], ks, 0);
    add_to_state<T, D, CT, NT>(W, cf, tb, b_lane, dec[half]);
    if (wave == 0 && i + 1 < chunks) decays(i + 1);
  };
  for (int i = 0; i < chunks; i += 2) {
    step(i, std::integral_constant<int, 0>());
    if (i + 1 < chunks) step(i + 1, std::integral_constant<int, 1>());
  }
  float* to = a.states + ((int64_t)slot * a.HV + h) * D * D;
#pragma unroll
  for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) *reinterpret_cast<f32x4*>(to + kept_at<D>(wave, kt, ct, lane)) = W[kt][ct];
  if (wave == 0) {
#pragma unroll
    for (int by = 32; by > 0; by >>= 1) sum += __shfl_xor(sum, by);
    // Rising log decays whose sums over a chunk are in FP32's range may leave it over a segment: a state of zeros stays one (a
    // test for zeros in the scan, or exponents apart from factors, cost it 1.4 us of 15.5 at 20,001 tokens and 8 heads)
    const float factor = __builtin_amdgcn_exp2f((float)(sum * 1.4426950408889634));
    if (lane == 0) a.decay[(int64_t)slot * a.HV + h] = factor > 0x1.fffffep127f ? 0x1.fffffep127f : factor;
  }
}

// Forward and, with n = 2 behind it in the same launch (`blocks` workgroups each), reverse. A launch of two dimensions has
// workgroups behind the last job's: these return before a job is chosen, which with n = 1 is the only one there is.
template <typename T, int D>
__global__ __launch_bounds__(NTHREADS, sizeof(T) == 2 ? 2 : 1) void k_linear_states(LinearJobs j, int blocks, int n) {
  const int b = block_index();
  if (b >= n * blocks) return;
  if (b < blocks) segment_state<T, D, false>(j.job[0], b);
  else segment_state<T, D, true>(j.job[1], b - blocks);
}

__device__ __forceinline__ double block_sum(double x, double* tmp) { // over 256 threads
#pragma unroll
  for (int by = 32; by > 0; by >>= 1) x += __shfl_xor(x, by);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
  __syncthreads();
  return (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
}

// The states that segments start from, in place of what they add: forward from `init` (h0) at the first segment,
// reverse from `init` (dht) at the last. In reverse, with `worth`: also this workgroup's part of <S, D> at the borders
// between segments, where S (`other`, from the forward scan) meets its gradient; see k_linear_dg. It costs moving the
// states (44 us for 265 MB), four of them ahead of the chain of sums.
template <int D, bool REV>
__global__ __launch_bounds__(256) void k_linear_scan(LinearArgs a, const float* other, double* worth) {
  constexpr int SIZE = D * D, PARTS = SIZE / 1024, AHEAD = 4;
  __shared__ double tmp[4];
  const int n = blockIdx.z, h = blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int from = cut_to(a.cu[n], a.T), to = max(cut_to(a.cu[n + 1], a.T), from);
  const int count = (to - from + a.seg - 1) / a.seg, base = doc_slot(a, n);
  const auto slot = [&](int i) { return base + (REV ? count - 1 - i : i); };
  const auto index = [&](int slot) { return ((int64_t)slot * a.HV + h) * SIZE + e; };
  f32x4 W = zero4();
  if (a.init && count > 1) {
    const float* p = a.init + ((int64_t)n * a.HV + h) * SIZE + kept_col<D>(e);
#pragma unroll
    for (int j = 0; j < 4; ++j) W[j] = p[(kept_row<D>(e) + j) * D];
  }
  for (int i = 0; i < count; i += AHEAD) {
    f32x4 add[AHEAD], meets[AHEAD];
    float dec[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      add[j] = meets[j] = zero4();
      dec[j] = 0.f;
      if (i + j < count - 1) {
        add[j] = *reinterpret_cast<const f32x4*>(a.states + index(slot(i + j)));
        dec[j] = a.decay[(int64_t)slot(i + j) * a.HV + h];
      }
      if (REV && worth && i + j < count && i + j > 0) meets[j] = *reinterpret_cast<const f32x4*>(other + index(slot(i + j) + 1));
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (i + j < count && i + j > 0) {
        *reinterpret_cast<f32x4*>(a.states + index(slot(i + j))) = W;
        if (REV && worth) {
          const f32x4 S = meets[j];
          const double x = block_sum(((double)S[0] * W[0] + (double)S[1] * W[1]) + ((double)S[2] * W[2] + (double)S[3] * W[3]), tmp);
          if (threadIdx.x == 0) worth[((int64_t)slot(i + j) * a.HV + h) * PARTS + blockIdx.x] = x;
        }
      }
      W = W * dec[j] + add[j];
    }
  }
}

// ------------------------------------------------------------------------------------------------
// The walk. A wave owns 16 CT columns of the state W (and of c and y) and keeps them in registers for the
// whole segment; a chunk takes
//   P    = decays * a b^T, its 16x16 tiles shared out to the waves, through LDS
//   y^T  = W^T a^T, each column times its row's factor       (W's registers are the operand as they are)
//   -- barrier: P is whole; a's and c's tiles are free, c is in registers
//   y^T += c^T P^T                                            (written out: 4 CT neighbouring columns a lane)
//   W    = decay W + b^T diag(w) c
//   -- barrier: the next tiles are there
// Four tiles in LDS: the next a goes where the last b was, at the chunk's start; the next b and c to where a and c
// were, after the first barrier. So each load has at least half a chunk to arrive, and two workgroups share a CU.
//
// P and W's operand are rounded once, to the io type: their products are summed in FP32 and the result is
// rounded to that type itself. So o and dv are off by 2.3e-3 where their own rounding alone leaves 1.7e-3; two terms for both
// would leave that, at 537 us for the forward of the tokens below instead of 470, 1930 for the backward instead of 1870, 91 for
// 20,001 tokens of 8 heads instead of 80 (f32 rows have none of these roundings). With DOTS (the decays' gradient, an FP32 result that is a difference of
// sums) both go in as EXACT terms instead. w c goes into W as EXACT terms where W is a result (DOTS, or the state that a
// document ends with), and as 2 where it is not: that leaves 2^-17 of each term, nothing beside W's own rounding
// (32,768 tokens, 48 heads, 128 wide, whole forward: one document 490 us, as 3 terms 504; four 495 and 500).
//
// Bound by the chain of a chunk's phases: some 130 matrix, 650 vector and 130 LDS instructions a wave in the forward, which two
// waves a SIMD overlap in small part. Of a SIMD's cycles in the backward's walks matrix instructions take 0.32 and vector
// instructions, 4 cycles each, up to 0.48 more (0.25 and 0.31 in the forward's, whose last workgroups leave CUs idle), at
// the 2.1 GHz that the card keeps through them. A third fewer matrix instructions in W's sum (above) gain 0 to 3%, a tenth fewer
// vector instructions 1.5% (the state's decay kept apart from W, which lost bits of ht and dg). The same 32,768
// tokens: forward 209 GFLOP of matrix instructions in 340 us, the backward's three 957 GFLOP in 1365 us.
template <typename T, int D>
struct WalkLds {
  static constexpr int P = 4 * Tile<T, D>::BYTES, P_TILE = 256;      // P: 10 tiles of 256 values
  static constexpr int dec(int p_size) { return P + 10 * P_TILE * p_size; } // Decays of two chunks
  static constexpr int red(int p_size) { return dec(p_size) + 2 * (int)sizeof(Decays); } // DOTS: [4 waves][64 rows]
  static constexpr int bytes(bool dots) { return red(dots ? 4 : sizeof(T)) + (dots ? 4 * CH * 4 : 0); }
};

// Parts of dq and dk, to be summed over a group's value heads (k_linear_group_sum): for bf16 as f16 multiples of a power
// of two that the 16 CT columns of a wave's row share, so that each keeps 11 bits, down to 2^-28 of the largest. That is
// off by 2^-12, a sixteenth of the sum's own rounding, and parts that cancel to a tenth still leave it that; bf16 parts
// would not. (32,768 tokens, 16/48 heads, 128 wide, whole backward: FP32 parts 2090 us, these 1934.)
// What is not finite makes its columns of the row NaN.
template <int CT>
struct PartRow {
  typedef _Float16 type __attribute__((ext_vector_type(4 * CT)));
};
template <int D, int CT>
__device__ __forceinline__ void write_part(const LinearArgs& a, const f32x4 (&y)[CT][4], int t, int n, int h, int wave) {
  const int lane = threadIdx.x & 63, g = fresh(lane >> 4), l16 = fresh(lane & 15), os = a.HV * D;
  const int64_t row = (int64_t)t * a.HV + h;
  const __amdgpu_buffer_rsrc_t to = make_rsrc((_Float16*)a.part + row * D, ((n - 1) * os + D) * 2);
  const __amdgpu_buffer_rsrc_t unit = make_rsrc(a.unit + row * 4, ((n - 1) * a.HV * 4 + 4) * 4);
  int off = (l16 * os + 16 * CT * wave + 4 * CT * g) * 2, uoff = (l16 * a.HV * 4 + wave) * 4;
#pragma unroll
  for (int bt = 0; bt < 4; ++bt, off += 32 * os, uoff += 256 * a.HV) {
    unsigned most = 0; // bits of magnitudes order as they do
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = y[ct][bt][e]; // a cast of the element itself would take the vector's first
        most = max(most, __builtin_bit_cast(unsigned, x) & 0x7fffffffu);
      }
    most = max(most, (unsigned)__shfl_xor((int)most, 16));
    most = max(most, (unsigned)__shfl_xor((int)most, 32));
    // 2^(exponent - 14), at least 2^-100, and its inverse, from the exponents' bits
    const int e = max((int)(most >> 23) - 14, 27);
    const float by = __builtin_bit_cast(float, (unsigned)(254 - e) << 23);
    typename PartRow<CT>::type v;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * ct + j] = (_Float16)(y[ct][bt][j] * by);
    if constexpr (CT == 2) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4_t, v), to, off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(i32x2_t, v), to, off, 0, 0);
    const float u = __builtin_bit_cast(float, most >= 0x7f800000u ? 0x7fc00000u : (unsigned)e << 23);
    if (g == 0) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, u), unit, uoff, 0, 0);
  }
}

template <typename T, int D, bool REV, bool DOTS, int NTW, typename F>
__device__ __forceinline__ void walk_chunks(const LinearArgs& a, const Segment& s, int h, f32x4 (&W)[D / 16][D / 64], const F& load_state) {
  typedef Tile<T, D> S;
  typedef Op<T> O;
  typedef typename O::frag frag;
  typedef WalkLds<T, D> L;
  constexpr int CT = D / 64, NT = DOTS ? O::EXACT : 1;
  typedef typename std::conditional<DOTS, float, T>::type PT; // type of P in LDS
  typedef PT p4 __attribute__((ext_vector_type(4)));
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int col0 = wave * 16 * CT;
  Decays* dec = (Decays*)(linear_lds + L::dec(sizeof(PT)));
  float* red = (float*)(linear_lds + L::red(sizeof(PT)));
  int ta = 0, tb = S::BYTES, spare = 2 * S::BYTES;
  constexpr int tc = 3 * S::BYTES;
  const int p_lane = L::P + lane * 4 * (int)sizeof(PT); // a lane reads of each tile what the same lane wrote

  const int chunks = (s.t1 - s.t0 + CH - 1) / CH;
  const auto at = [&](int i) { return s.t0 + (REV ? chunks - 1 - i : i) * CH; };
  const Feed<T, D> fa(a.a, a, h, wave), fb(a.b, a, h, wave), fc(a.c, a, h, wave);
  const int along = O::template along_lane<D>();
  const typename O::Down b_lane = O::template down_lane<D>(0, 4);
  typename O::Down c_lane[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) c_lane[ct] = O::template down_lane<D>(col0 + 4 * ct, 4 * CT);
  float gl = 0.f;
  const auto decays = [&](int i) { // of chunk i, and the log decays of the next
    chunk_decays<REV>(dec[i & 1], gl, a.in_scale, a.w_scale);
    gl = i + 1 < chunks ? log_decay(a, h, at(i + 1) + lane, s.t1) : 0.f;
  };
  fa.load(ta, at(0), s.t1);
  fb.load(tb, at(0), s.t1);
  fc.load(tc, at(0), s.t1);
  if (wave == 0) {
    gl = log_decay(a, h, at(0) + lane, s.t1);
    decays(0);
  }
  load_state();
  wait_loads<0>();
  for (int i = 0; i < chunks; ++i) {
    const int t = at(i), n = min(s.t1 - t, CH);
    const Decays& d = dec[i & 1];
    __syncthreads();
    const bool more = i + 1 < chunks;
    if (more) fa.load(spare, at(i + 1), s.t1);
    // P^T (rows s, column t) in tiles (x, z), z <= x: forward of rows x and columns z, in reverse the other way round.
    // Waves 0 and 1 take two of x = 3, wave 2 those of x = 2, wave 3 those of x = 1 and 0.
    {
      const int al = fresh(along), tx = REV ? tb : ta, tz = REV ? ta : tb;
      const int x = wave < 2 ? 3 : 4 - wave, z = wave == 1 ? 2 : 0;
      const auto finish = [&](const f32x4& p, int x, int z) {
        const int tt = 16 * (REV ? z : x) + l16, ss = 16 * (REV ? x : z) + 4 * g;
        const float th = d.hi[tt], tl = d.lo[tt];
        const f32x4 sh = *reinterpret_cast<const f32x4*>(&d.hi[ss]), sl = *reinterpret_cast<const f32x4*>(&d.lo[ss]);
        p4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x2 = REV ? (sh[j] - th) + (sl[j] - tl) : (th - sh[j]) + (tl - sl[j]);
          const bool keep = REV ? ss + j >= tt : ss + j <= tt;
          v[j] = (PT)(keep ? a.p_scale * p[j] * __builtin_amdgcn_exp2f(x2) : 0.f);
        }
        lds_write<p4>(p_lane + (x * (x + 1) / 2 + z) * L::P_TILE * (int)sizeof(PT), v);
      };
      const auto tile = [&](const frag& fx, const frag& fz, const f32x4& p) { return REV ? O::mul(fx, fz, p) : O::mul(fz, fx, p); };
      f32x4 p0 = zero4(), p1 = zero4();
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        const frag fx = O::template along<D>(tx, al, x, kk);
        p0 = tile(fx, O::template along<D>(tz, al, z, kk), p0);
        p1 = tile(fx, O::template along<D>(tz, al, z + 1, kk), p1);
      }
      finish(p0, x, z);
      finish(p1, x, z + 1);
      if (wave >= 2) {
        const int m = wave == 2 ? 2 : 0;
        f32x4 p2 = zero4();
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) p2 = tile(O::template along<D>(tx, al, m, kk), O::template along<D>(tz, al, m, kk), p2);
        finish(p2, m, m);
      }
    }
    frag cf[2][CT];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) cf[ks][ct] = O::template down<D>(tc, c_lane[ct], ks, 0);
    __builtin_amdgcn_s_setprio(1); // over the other workgroup's waves outside their products: 1 to 3% of the walk
    // y^T = W^T a^T
    const int al = fresh(along);
    f32x4 y[CT][4];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int bt = 0; bt < 4; ++bt) y[ct][bt] = zero4();
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
      frag af[4];
#pragma unroll
      for (int bt = 0; bt < 4; ++bt) af[bt] = O::template along<D>(ta, al, bt, kk);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const Terms<T, NT> w(join(W[2 * kk][ct], W[2 * kk + 1][ct]));
#pragma unroll
        for (int m = NT - 1; m >= 0; --m)
#pragma unroll
          for (int bt = 0; bt < 4; ++bt) y[ct][bt] = O::mul(w.f[m], af[bt], y[ct][bt]);
      }
    }
#pragma unroll
    for (int bt = 0; bt < 4; ++bt) {
      const float f = d.in[16 * bt + l16];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) y[ct][bt] *= f;
    }
    __builtin_amdgcn_s_setprio(0);
    __syncthreads(); // P
    __builtin_amdgcn_s_setprio(1);
    if (more) {
      fb.load(ta, at(i + 1), s.t1);
      fc.load(tc, at(i + 1), s.t1);
      if (wave == 0) decays(i + 1); // it has fewer tiles of P
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int bt = 0; bt < 4; ++bt) {
        if (REV ? ks < bt / 2 : ks > bt / 2) continue;
        const auto part = [&](int bs) -> p4 { // beside the diagonal: nothing
          if (REV ? bs < bt : bs > bt) return p4{(PT)0.f, (PT)0.f, (PT)0.f, (PT)0.f};
          const int x = REV ? bs : bt, z = REV ? bt : bs;
          return lds_read<p4>(p_lane + (x * (x + 1) / 2 + z) * L::P_TILE * (int)sizeof(PT));
        };
        const auto p8 = __builtin_shufflevector(part(2 * ks), part(2 * ks + 1), 0, 1, 2, 3, 4, 5, 6, 7);
        if constexpr (DOTS) {
          const Terms<T, NT> pf(p8);
#pragma unroll
          for (int m = NT - 1; m >= 0; --m)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) y[ct][bt] = O::mul(cf[ks][ct], pf.f[m], y[ct][bt]);
        } else {
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) y[ct][bt] = O::mul(cf[ks][ct], p8, y[ct][bt]);
        }
      }
    add_to_state<T, D, CT, NTW>(W, cf, tb, b_lane, d);

    __builtin_amdgcn_s_setprio(0);
    if constexpr (DOTS) {
#pragma unroll
      for (int bt = 0; bt < 4; ++bt) {
        const int row = 16 * bt + l16;
        const T* x = (const T*)a.dot.p + (int64_t)(t + min(row, n - 1)) * a.dot.stride + (int64_t)(a.dot.shared ? h / a.G : h) * D + col0 + 4 * CT * g;
        float sum = 0.f;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum = __builtin_fmaf((float)x[4 * ct + e], y[ct][bt][e], sum);
        sum = col_sum4(sum);
        if (g == 0) red[wave * CH + row] = sum;
      }
    }
    // y: lane (g, l16): row 16 bt + l16, columns col0 + 4 CT g ..; rows past the end lie past the buffer's, which drops them
    const auto write = [&](auto* out) {
      typedef typename std::remove_reference<decltype(*out)>::type Y;
      const int os = a.HV * D;
      const __amdgpu_buffer_rsrc_t to = make_rsrc(out + (int64_t)t * os + (int64_t)h * D, ((n - 1) * os + D) * (int)sizeof(Y));
      int off = (l16 * os + col0 + 4 * CT * g) * (int)sizeof(Y);
#pragma unroll
      for (int bt = 0; bt < 4; ++bt, off += 16 * os * (int)sizeof(Y)) {
        if constexpr (CT == 2 && sizeof(Y) == 2) {
          bf16x8 v;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = (bf16)y[e >> 2][bt][e & 3];
          buf_store16(v, to, off);
        } else {
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            const float v[4] = {y[ct][bt][0], y[ct][bt][1], y[ct][bt][2], y[ct][bt][3]};
            IO<Y>::bstore4(to, off / (int)sizeof(Y) + 4 * ct, v);
          }
        }
      }
    };
    if (a.part) {
      if constexpr (sizeof(T) == 4) {
        write((float*)a.part);
        wait_loads<4 * CT>(); // the next tiles, not these stores
      } else {
        write_part<D, CT>(a, y, t, n, h, wave);
        wait_loads<8>();
      }
    } else {
      write((T*)a.out);
      wait_loads<CT == 2 && sizeof(T) == 2 ? 4 : 4 * CT>();
    }
    if constexpr (DOTS) {
      __syncthreads();
      if ((int)threadIdx.x < n)
        a.dots[(int64_t)h * a.T + t + threadIdx.x] =
            (red[threadIdx.x] + red[CH + threadIdx.x]) + (red[2 * CH + threadIdx.x] + red[3 * CH + threadIdx.x]);
    }
    const int used = tb;
    tb = ta;
    ta = spare;
    spare = used;
  }
}

template <typename T, int D, bool REV, bool DOTS>
__device__ __forceinline__ void segment_walk(const LinearArgs& a, int block) {
  constexpr int CT = D / 64, EXACT = Op<T>::EXACT;
  int slot, h;
  if (!place(a, block, &slot, &h)) return;
  const Segment s = find_segment(a, slot);
  if (!s.live) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int col0 = wave * 16 * CT;
  const int64_t doc_state = ((int64_t)s.doc * a.HV + h) * D * D;
  const bool begins = REV ? s.last : s.first, ends = (REV ? s.first : s.last) && a.fin;

  // the state: rows 16 kt + 4 g + e, the lane's columns; `flip`: kept with rows and columns exchanged
  f32x4 W[D / 16][CT];
  const float* init = begins ? (a.init ? a.init + doc_state : nullptr) : nullptr;
  const float* kept = begins ? nullptr : a.states + ((int64_t)slot * a.HV + h) * D * D;
  const auto load_state = [&] {
#pragma unroll
    for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const int row = 16 * kt + 4 * g, col = column<CT>(col0, ct, l16);
        W[kt][ct] = zero4();
        if (kept) {
          if (!a.flip) W[kt][ct] = *reinterpret_cast<const f32x4*>(kept + kept_at<D>(wave, kt, ct, lane));
          else
#pragma unroll
            for (int e = 0; e < 4; ++e) W[kt][ct][e] = kept[kept_of<D>(col, row + e)];
        } else if (init) {
          if (a.flip) W[kt][ct] = *reinterpret_cast<const f32x4*>(init + col * D + row);
          else
#pragma unroll
            for (int e = 0; e < 4; ++e) W[kt][ct][e] = init[(row + e) * D + col];
        }
      }
  };
  if (s.t0 < s.t1) {
    if (DOTS || EXACT == 1 || ends) walk_chunks<T, D, REV, DOTS, EXACT>(a, s, h, W, load_state);
    else if constexpr (!DOTS && EXACT > 1) walk_chunks<T, D, REV, DOTS, 2>(a, s, h, W, load_state);
  } else load_state();
  if (ends) {
    float* to = a.fin + doc_state;
#pragma unroll
    for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int e = 0; e < 4; ++e) to[(16 * kt + 4 * g + e) * D + column<CT>(col0, ct, l16)] = W[kt][ct][e];
  }
}

template <typename T, int D>
__global__ __launch_bounds__(NTHREADS, sizeof(T) == 2 ? 2 : 1) void k_linear_walk(LinearArgs a) {
  segment_walk<T, D, false, false>(a, block_index());
}
// The backward's three in one launch, `blocks` workgroups each: dq, dk, dv. What a launch of two dimensions has behind them
// (here and in the forward's walk) is refused by place(): its slot is past the last.
template <typename T, int D, bool DOTS>
__global__ __launch_bounds__(NTHREADS, sizeof(T) == 2 ? 2 : 1) void k_linear_walks(LinearJobs j, int blocks) {
  const int b = block_index();
  if (b < blocks) segment_walk<T, D, false, DOTS>(j.job[0], b);
  else if (b < 2 * blocks) segment_walk<T, D, true, DOTS>(j.job[1], b - blocks);
  else segment_walk<T, D, true, false>(j.job[2], b - 2 * blocks);
}

// ------------------------------------------------------------------------------------------------
// Sums over the value heads of a group, in their order and in FP32: part [T, HV, D] -> out [T, H, D], for dq and dk, but
// for rows of no document, whose parts nobody wrote. It costs moving the parts: 1.1 GB of 16-bit ones at 32,768 tokens,
// 16/48 heads, 128 wide take 196 us (FP32 ones 355).
template <typename T, int D>
__global__ __launch_bounds__(256) void k_linear_group_sum(LinearJobs jobs) {
  const LinearArgs& a = jobs.job[blockIdx.y];
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8, n = (int64_t)a.T * a.H * D;
  if (i >= n) return;
  const int64_t row = i / D; // of [T, H]
  if (row < (int64_t)cut_to(a.cu[0], a.T) * a.H || row >= (int64_t)cut_to(a.cu[a.N], a.T) * a.H) return;
  const int64_t head = row * a.G;
  const int col = (int)(i % D);
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.f;
  for (int j = 0; j < a.G; ++j) {
    const int64_t at = (head + j) * D + col;
    if constexpr (sizeof(T) == 4) {
      float x[8];
      IO<float>::load8f((const float*)a.part + at, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += x[e];
    } else {
      const auto x = *reinterpret_cast<const PartRow<2>::type*>((const _Float16*)a.part + at);
      const float u = a.unit[(head + j) * 4 + col / (D / 4)];
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf((float)x[e], u, s[e]);
    }
  }
  IO<T>::store4((T*)a.out + i, s);
  IO<T>::store4((T*)a.out + i + 4, s + 4);
}

// ------------------------------------------------------------------------------------------------
// The decays' gradient. The differences q.dq - k.dk cancel to a large part, and summed over a whole document their
// roundings would outgrow what is left. So each segment is summed by itself, between borders where the gradient is known
// apart from those sums: it is <S, D> of the state there and its own gradient, which the scan in reverse has summed. With
// n tokens, sums from the end and E = <S, D> at the end, dg_t = E + sum_{s >= t} (q_s.dq_s - k_s.dk_s), and at the first
// token that has to be <S, D> at the start: what it misses is spread evenly over the tokens, which leaves a
// third of the roundings. At a document's start S is h0 or 0; at its end D is 0, or with dht S is not at hand, and
// the sum runs from the start alone. Where the factor e^g itself is 0 in FP32 (g below the logarithm of half its smallest
// number) so is dg_t = e^g <S, D>: written as 0, where the sums leave their roundings.
__global__ __launch_bounds__(256) void k_linear_dg(LinearDgArgs d) {
  const LinearArgs& a = d.a;
  __shared__ double tmp[4], carry[4];
  const int slot = blockIdx.x, h = blockIdx.y, size = a.D * a.D, parts = size / 1024;
  const Segment s = find_segment(a, slot);
  const int n = s.live ? s.t1 - s.t0 : 0;
  const float *qd = d.qdots + (int64_t)h * a.T + s.t0, *kd = d.kdots + (int64_t)h * a.T + s.t0;
  const auto border = [&](int slot) { // behind that segment
    double x = 0.0;
    if ((int)threadIdx.x < parts) x = d.worth[((int64_t)slot * a.HV + h) * parts + threadIdx.x];
    return block_sum(x, tmp);
  };
  double start = 0.0, end = 0.0, all = 0.0;
  bool from_end = true;
  if (n > 0) {
    if (!s.first) start = border(slot - 1);
    else if (d.h0) {
      const int64_t at = ((int64_t)s.doc * a.HV + h) * size;
      double x = 0.0;
      for (int e = threadIdx.x * 4; e < size; e += 1024) {
        const f32x4 u = *reinterpret_cast<const f32x4*>(d.h0 + at + e), v = *reinterpret_cast<const f32x4*>(d.dh0 + at + e);
        x += ((double)u[0] * v[0] + (double)u[1] * v[1]) + ((double)u[2] * v[2] + (double)u[3] * v[3]);
      }
      start = block_sum(x, tmp);
    }
    if (!s.last) end = border(slot);
    from_end = !(s.last && d.dht);
  }
  double spread = 0.0; // what each token takes of what is missed
  if (from_end && n > 0) {
    double x = 0.0;
    for (int t = threadIdx.x; t < n; t += 256) x += (double)qd[t] - (double)kd[t];
    spread = (start - (end + block_sum(x, tmp))) / n;
  }
  double f = from_end ? end : start;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int c = 0; c < n; c += 256) { // from the border inwards
    const int j = c + (int)threadIdx.x, t = from_end ? n - 1 - j : j;
    const double own = j < n ? (double)qd[t] - (double)kd[t] : 0.0;
    const float g = j < n ? log_decay(a, h, s.t0 + t, s.t1) : 0.f;
    const double p = wave_sums(own);
    if (lane == 63) carry[wave] = p;
    __syncthreads();
    double before = 0.0, turn = 0.0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      before += w < wave ? carry[w] : 0.0;
      turn += carry[w];
    }
    double v = from_end ? f + before + p + spread * (j + 1) : f - before - (p - own);
    if (j < n) {
      if (g < -104.f) v = 0.0;
      if (a.gs) d.dg[(int64_t)(s.t0 + t) * a.HV + h] = (float)v;
      all += v;
    }
    f += from_end ? turn : -turn;
    __syncthreads();
  }
  if (a.gs == 0) { // one decay a head: the sum of dg over the segment
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

template <typename T, int D>
static int states_t(const LinearJobs& j, int n, hipStream_t s) {
  constexpr unsigned lds = 4 * Tile<T, D>::BYTES + 2 * sizeof(Decays);
  static std::atomic<uint64_t> asked{0};
  if (const int e = ask_lds(reinterpret_cast<const void*>(&k_linear_states<T, D>), lds, asked)) return e;
  const unsigned blocks = place_blocks(j.job[0]);
  hipLaunchKernelGGL((k_linear_states<T, D>), many_blocks(blocks * n), dim3(NTHREADS), lds, s, j, (int)blocks, n);
  return (int)hipGetLastError();
}
template <typename T, int D>
static int walk_t(const LinearArgs& a, hipStream_t s) {
  constexpr unsigned lds = WalkLds<T, D>::bytes(false);
  static std::atomic<uint64_t> asked{0};
  if (const int e = ask_lds(reinterpret_cast<const void*>(&k_linear_walk<T, D>), lds, asked)) return e;
  hipLaunchKernelGGL((k_linear_walk<T, D>), many_blocks(place_blocks(a)), dim3(NTHREADS), lds, s, a);
  return (int)hipGetLastError();
}
template <typename T, int D, bool DOTS>
static int walks_t(const LinearJobs& j, hipStream_t s) {
  constexpr unsigned lds = WalkLds<T, D>::bytes(DOTS);
  static std::atomic<uint64_t> asked{0};
  if (const int e = ask_lds(reinterpret_cast<const void*>(&k_linear_walks<T, D, DOTS>), lds, asked)) return e;
  const unsigned blocks = place_blocks(j.job[0]);
  hipLaunchKernelGGL((k_linear_walks<T, D, DOTS>), many_blocks(3 * blocks), dim3(NTHREADS), lds, s, j, (int)blocks);
  return (int)hipGetLastError();
}
template <typename T, int D>
static int walks_td(const LinearJobs& j, hipStream_t s) {
  return j.job[0].dots ? walks_t<T, D, true>(j, s) : walks_t<T, D, false>(j, s);
}

int launch_linear_states(const LinearJobs& j, int n, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool wide = j.job[0].D == 128;
  if (dtype == 0) return wide ? states_t<bf16, 128>(j, n, s) : states_t<bf16, 64>(j, n, s);
  return wide ? states_t<float, 128>(j, n, s) : states_t<float, 64>(j, n, s);
}

int launch_linear_scan(const LinearArgs& a, bool rev, const float* other, double* worth, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(a.D * a.D / 1024), (unsigned)a.HV, (unsigned)a.N);
  if (a.D == 128) {
    if (rev) hipLaunchKernelGGL((k_linear_scan<128, true>), grid, dim3(256), 0, s, a, other, worth);
    else hipLaunchKernelGGL((k_linear_scan<128, false>), grid, dim3(256), 0, s, a, other, worth);
  } else {
    if (rev) hipLaunchKernelGGL((k_linear_scan<64, true>), grid, dim3(256), 0, s, a, other, worth);
    else hipLaunchKernelGGL((k_linear_scan<64, false>), grid, dim3(256), 0, s, a, other, worth);
  }
  return (int)hipGetLastError();
}

int launch_linear_walk(const LinearArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == 0) return a.D == 128 ? walk_t<bf16, 128>(a, s) : walk_t<bf16, 64>(a, s);
  return a.D == 128 ? walk_t<float, 128>(a, s) : walk_t<float, 64>(a, s);
}

int launch_linear_walks(const LinearJobs& j, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool wide = j.job[0].D == 128;
  if (dtype == 0) return wide ? walks_td<bf16, 128>(j, s) : walks_td<bf16, 64>(j, s);
  return wide ? walks_td<float, 128>(j, s) : walks_td<float, 64>(j, s);
}

int launch_linear_group_sum(const LinearJobs& j, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int64_t n = (int64_t)j.job[0].T * j.job[0].H * j.job[0].D / 8;
  if (n == 0) return 0;
  const dim3 grid((unsigned)((n + 255) / 256), 2);
  if (j.job[0].D == 128) {
    if (dtype == 0) hipLaunchKernelGGL((k_linear_group_sum<bf16, 128>), grid, dim3(256), 0, s, j);
    else hipLaunchKernelGGL((k_linear_group_sum<float, 128>), grid, dim3(256), 0, s, j);
  } else {
    if (dtype == 0) hipLaunchKernelGGL((k_linear_group_sum<bf16, 64>), grid, dim3(256), 0, s, j);
    else hipLaunchKernelGGL((k_linear_group_sum<float, 64>), grid, dim3(256), 0, s, j);
  }
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
