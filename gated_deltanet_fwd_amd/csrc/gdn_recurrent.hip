// The gated delta rule, recurrent, on cached FP32 states (gfx950): one token a sequence when
// decoding, short runs when drafted tokens are checked or a prompt is extended. Per token and
// value head, with a = exp(g), raw rows k and q and their inverse norms rk, rq (1 without the norm):
//
//   s1 = S^T k,  s2 = S^T q                  (one pass over the old state)
//   u  = beta rk (v - a rk s1)
//   o  = rq (a s2 + (q.k) u)                 (= rq S_new^T q)
//   S  = a S + k u^T
//
// Columns of S (value indices) never mix, so a wave owns some columns of one head's state and keeps
// them in registers from the first token to the last. Two kernels: k_recurrent_step for calls bound
// by moving the states, k_recurrent_run for longer runs, bound by the chain from token to token.
#include "gdn_device.h"

namespace gdn {

constexpr unsigned MAX_GRID_Y = 65535;

template <typename T, int N>
struct Vec {
  typedef T type __attribute__((ext_vector_type(N)));
};
template <typename T>
struct Vec<T, 1> {
  typedef T type;
};

template <typename T, int N>
__device__ __forceinline__ void unpack(const typename Vec<T, N>::type& r, float* v) {
  if constexpr (N == 1) v[0] = (float)r;
  else
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = (float)r[e];
}

__device__ __forceinline__ float lane_value(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// The lane-swap instructions exchange the odd 16-lane rows (swap16) or the upper half (swap32) of x
// with the even rows or the lower half of y.
struct Pair {
  float x, y;
};
__device__ __forceinline__ Pair swap16(float x, float y) {
  const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y), false, false);
  return {__builtin_bit_cast(float, (unsigned)s[0]), __builtin_bit_cast(float, (unsigned)s[1])};
}
__device__ __forceinline__ Pair swap32(float x, float y) {
  const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y), false, false);
  return {__builtin_bit_cast(float, (unsigned)s[0]), __builtin_bit_cast(float, (unsigned)s[1])};
}
// x in a register of its own (with one value as both operands the compiler folds a swap away)
__device__ __forceinline__ float copy_of(float x) {
  asm("" : "+v"(x));
  return x;
}

// The wave's place in a grid of (heads x blocks of columns / 4, sequences); cb counts within a state.
__device__ __forceinline__ bool wave_of(const RecurrentArgs& a, int blocks, int* n, int* h, int* j, int* cb) {
  const int w = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  *n = (int)(blockIdx.z * MAX_GRID_Y + blockIdx.y);
  *h = w / blocks;
  *cb = w % blocks;
  *j = (int)(((uint64_t)*h * a.g_mul) >> 32);
  return *h < a.HV && *n < a.N;
}

// cache policies of a buffer access: non-temporal; non-temporal and written through
constexpr int NT = 2, WRITE_THROUGH = 19;

// ------------------------------------------------------------------------------------------------
// One token, or a few: a wave holds 32 columns, lane (kg, cg) = (lane / 8, lane % 8) the D / 8 keys
// from kg D / 8 on of columns 4 cg .. 4 cg + 3, so a load or store covers whole 128-byte lines.
// What it costs is moving the states. They are read and written non-temporally: they are not used
// again before the next step, and the same pattern without it moves a tenth less. With one token a
// sequence each row of the new state leaves as it is made, and few waves share a CU: a workgroup asks
// for STEP_LDS bytes of LDS that it does not use, which leaves two a CU, and the compiler is told to
// use the registers of 3 waves a SIMD. 128 KB of states in flight are enough, and more only get in
// each other's way. 256 sequences at 48 heads, 128 wide (805 MB each way): 269-275 us, 5.9-6.0 TB/s,
// as an in-place elementwise pass over such a buffer; 294 us without these. 8 sequences: 9.1 us
// instead of 10.8. With slot_tok the call mostly writes, and writing through gains another 5%: 24
// sequences of up to 8 tokens, 352 MB, 69 us instead of 72. Absent states are buffers of no bytes:
// loads give zeros, stores are dropped, and no branch stands between loads and their use.
constexpr unsigned STEP_LDS = 64 * 1024;

enum StepKind { ONE_TOKEN, RUN_OF_TOKENS, KEEP_EACH }; // one token a sequence; several; with slot_tok

template <typename TI, int D, StepKind KIND>
__global__ __launch_bounds__(256)
__attribute__((amdgpu_waves_per_eu(KIND == ONE_TOKEN ? 3 : 1, KIND == ONE_TOKEN ? 3 : 8))) void k_recurrent_step(RecurrentArgs a) {
  constexpr int KPL = D / 8, CB = D / 32;
  typedef typename Vec<TI, KPL>::type kvec;
  const int lane = threadIdx.x & 63, cg = lane & 7, kg = lane >> 3;
  int n, h, j, cb; // sequence, value head, q/k head, block of columns
  if (!wave_of(a, CB, &n, &h, &j, &cb)) return;
  cb *= 32;
  // after the sums over the keys a lane keeps the totals of one column, 2 (lane / 32) + lane / 16 % 2
  // of its four, and the value and output of that column
  const int col = cb + 4 * cg + 2 * (lane >> 5) + ((lane >> 4) & 1);
  const bool writes = !(lane & 8);
  TI* o = (TI*)a.o + (int64_t)h * D + col;
  const int64_t os = (int64_t)a.HV * D;
  const SeqSpan sp = seq_span(a.cu, a.slot_in, a.slot_out, n, a.T, a.n_slots);
  const float nan = __builtin_nanf("");
  if (!sp.ok) {
    for (int t = sp.t0; t < sp.t1; ++t)
      if (writes) o[t * os] = (TI)nan;
    return;
  }
  const int64_t hd = (int64_t)a.HV * D * D, head = (int64_t)h * D * D;
  const int at = 4 * (kg * KPL * D + cb + 4 * cg); // bytes
  const auto state = [&](int slot) {
    return make_rsrc(a.states + (slot < 0 ? 0 : slot) * hd + head, slot < 0 ? 0 : D * D * 4);
  };
  f32x4 S[KPL];
  const __amdgpu_buffer_rsrc_t from = state(sp.in);
#pragma unroll
  for (int i = 0; i < KPL; ++i)
    S[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, at + 4 * D * i, 0, NT));
  const auto store_row = [&](const __amdgpu_buffer_rsrc_t& to, int i) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4_t, S[i]), to, at + 4 * D * i, 0, KIND == KEEP_EACH ? WRITE_THROUGH : NT);
  };
  struct Rows {
    kvec k, q;
    TI v;
    float g, beta;
    int st;
  };
  const TI* qp = (const TI*)a.q + (int64_t)j * D + kg * KPL;
  const TI* kp = (const TI*)a.k + (int64_t)j * D + kg * KPL;
  const TI* vp = (const TI*)a.v + (int64_t)h * D + col;
  const auto load = [&](Rows& r, int t) {
    r.k = *reinterpret_cast<const kvec*>(kp + t * a.ks);
    r.q = *reinterpret_cast<const kvec*>(qp + t * a.qs);
    r.v = vp[t * a.vs];
    r.g = a.g[(int64_t)t * a.HV + h];
    r.beta = a.beta[(int64_t)t * a.HV + h];
    if constexpr (KIND == KEEP_EACH) r.st = a.slot_tok[t];
  };
  const auto all = [](float x) { // sum over the key groups, in every lane
    x += dpp<0x128>(x);
    Pair p = swap16(x, copy_of(x));
    p = swap32(p.x + p.y, copy_of(p.x + p.y));
    return p.x + p.y;
  };
  const auto compute = [&](const Rows& r, int t) {
    float kf[KPL], qf[KPL];
    unpack<TI, KPL>(r.k, kf);
    unpack<TI, KPL>(r.q, qf);
    float kk = 0.f, qq = 0.f, qk = 0.f;
    f32x4 s1 = zero4(), s2 = zero4();
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      kk = __builtin_fmaf(kf[i], kf[i], kk);
      qq = __builtin_fmaf(qf[i], qf[i], qq);
      qk = __builtin_fmaf(qf[i], kf[i], qk);
    }
    const float rk = a.l2norm ? inv_sqrt(all(kk) + 1e-6f) : 1.f;
    const float rq = a.l2norm ? inv_sqrt(all(qq) + 1e-6f) : 1.f;
    qk = all(qk);
    const float al = __expf(r.g);
#pragma unroll
    for (int i = 0; i < KPL; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s1[c] = __builtin_fmaf(S[i][c], kf[i], s1[c]);
        s2[c] = __builtin_fmaf(S[i][c], qf[i], s2[c]);
      }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      s1[c] += dpp<0x128>(s1[c]);
      s2[c] += dpp<0x128>(s2[c]);
    }
    Pair x0 = swap32(s1[0], s1[2]), x1 = swap32(s1[1], s1[3]);
    Pair y0 = swap32(s2[0], s2[2]), y1 = swap32(s2[1], s2[3]);
    x0 = swap16(x0.x + x0.y, x1.x + x1.y);
    y0 = swap16(y0.x + y0.y, y1.x + y1.y);
    const float u = r.beta * rk * __builtin_fmaf(-al * rk, x0.x + x0.y, (float)r.v);
    float out = rq * __builtin_fmaf(al, y0.x + y0.y, qk * u);
    int keep = -1;
    if constexpr (KIND == ONE_TOKEN) keep = sp.out;
    if constexpr (KIND == KEEP_EACH) {
      const bool bad = r.st < -1 || r.st >= a.n_slots;
      keep = bad ? -1 : r.st;
      out = bad ? nan : out;
    }
    if (writes) o[t * os] = (TI)out;
    // the four columns' u in every lane
    const Pair w = swap16(u, copy_of(u));
    const Pair w0 = swap32(w.x, copy_of(w.x)), w1 = swap32(w.y, copy_of(w.y));
    const f32x4 uu = {w0.x, w1.x, w0.y, w1.y};
    const __amdgpu_buffer_rsrc_t to = state(keep);
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) S[i][c] = __builtin_fmaf(kf[i], uu[c], al * S[i][c]);
      if constexpr (KIND != RUN_OF_TOKENS) {
        store_row(to, i);
        __builtin_amdgcn_sched_barrier(0); // each row leaves as it is made, not all of them at the end
      }
    }
  };
  if constexpr (KIND == ONE_TOKEN) {
    Rows r;
    load(r, sp.t0);
    compute(r, sp.t0);
  } else {
    const int last = sp.t1 - 1;
    if (sp.t0 <= last) {
      Rows x, y;
      load(x, sp.t0);
      for (int t = sp.t0; t <= last; t += 2) {
        load(y, min(t + 1, last));
        compute(x, t);
        if (t == last) break;
        load(x, min(t + 2, last));
        compute(y, t + 1);
      }
    }
    const __amdgpu_buffer_rsrc_t to = state(sp.out);
#pragma unroll
    for (int i = 0; i < KPL; ++i) store_row(to, i);
  }
}

// ------------------------------------------------------------------------------------------------
// Runs: what bounds them is issuing each token's instructions in turn (few sequences: one wave a SIMD,
// about 60 instructions a token; many: the 3 operations of each state element and token). A state is
// spread over more waves and the keys' sums go through DPP adds, which leave the total in every lane. Lane (c, kk) =
// (lane / 16, lane % 16) holds the D / 16 keys from kk D / 16 on of CPL columns; a wave holds 4 CPL.
// Tokens are taken 4 at a time: the rows of the next 4 are loaded while these are computed, lane row
// c makes the norms, q.k and gates of token c, and the 4 outputs leave in one store.
// The decay is kept as a factor f of the whole state (S = f R: R += k (u / f)^T), one operation less
// for each state element and token; R takes it over when f would leave [2^-24, 2^24].
template <typename TI, int D, int CPL, bool TOK>
__global__ __launch_bounds__(256) void k_recurrent_run(RecurrentArgs a) {
  constexpr int KPL = D / 16, CB = D / (4 * CPL), U = 4;
  typedef typename Vec<TI, KPL>::type kvec;
  typedef typename Vec<TI, CPL>::type vvec;
  typedef typename Vec<float, CPL>::type svec;
  const int lane = threadIdx.x & 63, kk = lane & 15, c = lane >> 4;
  int n, h, j, cb; // sequence, value head, q/k head, block of columns
  if (!wave_of(a, CB, &n, &h, &j, &cb)) return;
  const int col = (cb * 4 + c) * CPL;
  const int os = a.HV * D;
  const SeqSpan sp = seq_span(a.cu, a.slot_in, a.slot_out, n, a.T, a.n_slots);
  const float nan = __builtin_nanf("");
  if (!sp.ok) {
    for (int t = sp.t0 + kk; t < sp.t1; t += 16)
      for (int e = 0; e < CPL; ++e) ((TI*)a.o)[(int64_t)t * os + h * D + col + e] = (TI)nan;
    return;
  }
  const int64_t hd = (int64_t)a.HV * D * D, head = (int64_t)h * D * D;
  const int at = kk * KPL * D + col;
  float S[KPL][CPL];
  {
    const float* p = a.states + (sp.in < 0 ? 0 : sp.in) * hd + head + at;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      unpack<float, CPL>(*reinterpret_cast<const svec*>(p + i * D), S[i]);
#pragma unroll
      for (int e = 0; e < CPL; ++e) S[i][e] = keepf(S[i][e], sp.in >= 0);
    }
  }
  float f = 1.f;
  const auto store_state = [&](int slot) {
    float* p = a.states + slot * hd + head + at;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      svec r;
      if constexpr (CPL == 1) r = f * S[i][0];
      else
#pragma unroll
        for (int e = 0; e < CPL; ++e) r[e] = f * S[i][e];
      *reinterpret_cast<svec*>(p + i * D) = r;
    }
  };
  struct Block {
    kvec k[U], q[U], kn, qn;
    vvec v;
    float g, beta;
    int st;
  };
  const int t0 = sp.t0, last = sp.t1 - 1;
  // row offsets inside a block of tokens are 32-bit (the host checks the strides)
  const int ks = (int)a.ks, qs = (int)a.qs, vs = (int)a.vs, ko = j * D + kk * KPL, vo = h * D + col;
  // Rows of the block of tokens t .. t + 3, cut at the last token. With one column a lane a token is
  // about 40 instructions, and the addresses of its rows are kept and moved on by a block (147 ns a
  // token instead of 183, 64 wide, f32); with four they are made for each block, and the two paths of
  // `compute` are one, to leave the registers to the waves (323 us instead of 349 for 12 sequences of
  // up to 300 tokens of 48 heads).
  constexpr bool KEPT = CPL == 1;
  struct Rows {
    const TI *k[U], *q[U], *kn, *qn, *v;
    const float *g, *beta;
    const int32_t* st;
  } at_rows;
  const auto rows_of = [&](Rows& r, int t) {
    const int lim = last - t, tc = min(c, lim);
    const TI* kp = (const TI*)a.k + (int64_t)t * a.ks;
    const TI* qp = (const TI*)a.q + (int64_t)t * a.qs;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r.k[u] = kp + (ko + min(u, lim) * ks);
      r.q[u] = qp + (ko + min(u, lim) * qs);
    }
    r.kn = kp + (ko + tc * ks);
    r.qn = qp + (ko + tc * qs);
    r.v = (const TI*)a.v + (int64_t)t * a.vs + (vo + min(kk & 3, lim) * vs);
    r.g = a.g + ((int64_t)t * a.HV + h) + tc * a.HV;
    r.beta = a.beta + ((int64_t)t * a.HV + h) + tc * a.HV;
    r.st = TOK ? a.slot_tok + t + tc : nullptr;
  };
  const auto load = [&](Block& b, int t) {
    if constexpr (!KEPT) rows_of(at_rows, min(t, last));
    Rows& r = at_rows;
    b.kn = *reinterpret_cast<const kvec*>(r.kn);
    b.qn = *reinterpret_cast<const kvec*>(r.qn);
    b.g = *r.g;
    b.beta = *r.beta;
    b.v = *reinterpret_cast<const vvec*>(r.v);
    if constexpr (TOK) b.st = *r.st;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      b.k[u] = *reinterpret_cast<const kvec*>(r.k[u]);
      b.q[u] = *reinterpret_cast<const kvec*>(r.q[u]);
    }
    if constexpr (KEPT) {
      if (t + 2 * U - 1 <= last) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          r.k[u] += U * ks;
          r.q[u] += U * qs;
        }
        r.kn += U * ks;
        r.qn += U * qs;
        r.v += U * vs;
        r.g += U * a.HV;
        r.beta += U * a.HV;
        if constexpr (TOK) r.st += U;
      } else {
        rows_of(r, min(t + U, last));
      }
    }
  };
  // one token of a block; f is the factor of R with its decay
  const auto token = [&](const Block& b, int u, float rq, float qk, float b1, float b2, const float vf[CPL],
                         float held[CPL]) {
    float kf[KPL], qf[KPL], s1[CPL], s2[CPL];
    unpack<TI, KPL>(b.k[u], kf);
    unpack<TI, KPL>(b.q[u], qf);
    const float c1 = lane_value(b1, 16 * u) * __builtin_amdgcn_rcpf(f), c2 = lane_value(b2, 16 * u);
    const float qku = lane_value(qk, 16 * u), fq = f * lane_value(rq, 16 * u);
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
      s1[e] = S[0][e] * kf[0];
      s2[e] = S[0][e] * qf[0];
#pragma unroll
      for (int i = 1; i < KPL; ++i) {
        s1[e] = __builtin_fmaf(S[i][e], kf[i], s1[e]);
        s2[e] = __builtin_fmaf(S[i][e], qf[i], s2[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
      const float v = u == 0 ? dpp<0x150>(vf[e]) : u == 1 ? dpp<0x151>(vf[e]) : u == 2 ? dpp<0x152>(vf[e]) : dpp<0x153>(vf[e]);
      const float w = __builtin_fmaf(-c2, row_sum16(s1[e]), c1 * v); // u / f
      const float out = fq * __builtin_fmaf(qku, w, row_sum16(s2[e]));
      held[e] = kk == u ? out : held[e];
#pragma unroll
      for (int i = 0; i < KPL; ++i) S[i][e] = __builtin_fmaf(kf[i], w, S[i][e]);
    }
    if constexpr (TOK) {
      const int st = __builtin_amdgcn_readlane(b.st, 16 * u);
      if (st < -1 || st >= a.n_slots) {
#pragma unroll
        for (int e = 0; e < CPL; ++e) held[e] = kk == u ? nan : held[e];
      } else if (st >= 0) {
        store_state(st);
      }
    }
  };
  const auto compute = [&](const Block& b, int t, int count) {
    // of token c of the block, in lane row c
    float rk = 1.f, rq = 1.f, qk = 0.f, vf[CPL], kf[KPL], qf[KPL], held[CPL];
    unpack<TI, KPL>(b.kn, kf);
    unpack<TI, KPL>(b.qn, qf);
#pragma unroll
    for (int i = 0; i < KPL; ++i) qk = __builtin_fmaf(qf[i], kf[i], qk);
    qk = row_sum16(qk);
    if (a.l2norm) {
      float ss = 0.f, qq = 0.f;
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        ss = __builtin_fmaf(kf[i], kf[i], ss);
        qq = __builtin_fmaf(qf[i], qf[i], qq);
      }
      rk = inv_sqrt(row_sum16(ss) + 1e-6f);
      rq = inv_sqrt(row_sum16(qq) + 1e-6f);
    }
    const float b1 = b.beta * rk, b2 = b1 * rk, al = __expf(b.g);
    unpack<TI, CPL>(b.v, vf);
    float fu[U], lo = f, hi = f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      fu[u] = (u ? fu[u - 1] : f) * lane_value(al, 16 * u);
      lo = fminf(lo, fu[u]);
      hi = fmaxf(hi, fu[u]);
    }
    const bool in = lo >= 5.9604645e-8f && hi <= 1.6777216e7f; // a NaN passes, and its state is NaN either way
    if (KEPT && count == U && in) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f = fu[u];
        token(b, u, rq, qk, b1, b2, vf, held);
      }
    } else { // a block cut short, decays that have to go into the state token by token, or several columns
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= count) break;
        if (KEPT || !in) {
          const float x = f * lane_value(al, 16 * u);
#pragma unroll
          for (int i = 0; i < KPL; ++i)
#pragma unroll
            for (int e = 0; e < CPL; ++e) S[i][e] *= x;
          f = 1.f;
        } else {
          f = fu[u];
        }
        token(b, u, rq, qk, b1, b2, vf, held);
      }
    }
    if (kk < count) {
      vvec r;
      if constexpr (CPL == 1) r = (TI)held[0];
      else
#pragma unroll
        for (int e = 0; e < CPL; ++e) r[e] = (TI)held[e];
      *reinterpret_cast<vvec*>((TI*)a.o + (int64_t)t * os + (kk * os + vo)) = r;
    }
  };
  if (t0 <= last) {
    Block x, y;
    if constexpr (KEPT) rows_of(at_rows, t0);
    load(x, t0);
    for (int t = t0; t <= last; t += 2 * U) {
      load(y, t + U);
      compute(x, t, min(U, last + 1 - t));
      if (t + U > last) break;
      load(x, t + 2 * U);
      compute(y, t + U, min(U, last + 1 - t - U));
    }
  }
  if (sp.out >= 0) store_state(sp.out);
}

static dim3 grid_of(const RecurrentArgs& a, int waves_per_state) {
  const unsigned n = (unsigned)a.N;
  return dim3((unsigned)((a.HV * waves_per_state + 3) / 4), n < MAX_GRID_Y ? n : MAX_GRID_Y,
              (n + MAX_GRID_Y - 1) / MAX_GRID_Y);
}

template <typename TI, int D, int CPL>
static void run_c(const RecurrentArgs& a, hipStream_t s) {
  const dim3 grid = grid_of(a, D / (4 * CPL));
  if (a.slot_tok) hipLaunchKernelGGL((k_recurrent_run<TI, D, CPL, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_recurrent_run<TI, D, CPL, false>), grid, dim3(256), 0, s, a);
}

// The kernel by the longest sequence, as the host knows it. Up to 6 tokens the step is no slower, from
// 8 on the run is faster (16 heads of 48, 128 wide, us step / run: 1 sequence of 4 tokens 7.6 / 8.9,
// of 8 11.3 / 10.7, of 16 18.9 / 13.5; 32 sequences 42.0 / 42.3, 55.8 / 51.0, 88.9 / 79.0). With every
// state kept the step's stores are the better ones for longer (8 sequences of 16 tokens 81 / 116).
// A run takes four columns a lane once that gives 512 waves, one below (us for 200 tokens, one / four
// columns: 1 sequence 78 / 96, 2 sequences, 768 waves, 109 / 98, 8 sequences 351 / 224).
template <typename TI, int D>
static int recurrent_t(const RecurrentArgs& a, hipStream_t s) {
  const int64_t waves4 = (int64_t)a.live * a.HV * (D / 16); // of a run at four columns a lane
  const dim3 step = grid_of(a, D / 32);
  if (!a.cu && !a.slot_tok) {
    hipLaunchKernelGGL((k_recurrent_step<TI, D, ONE_TOKEN>), step, dim3(256), STEP_LDS, s, a);
  } else if (a.slot_tok && a.longest <= 32) {
    hipLaunchKernelGGL((k_recurrent_step<TI, D, KEEP_EACH>), step, dim3(256), STEP_LDS, s, a);
  } else if (a.longest <= 6) {
    hipLaunchKernelGGL((k_recurrent_step<TI, D, RUN_OF_TOKENS>), step, dim3(256), STEP_LDS, s, a);
  } else if (waves4 >= 512) {
    run_c<TI, D, 4>(a, s);
  } else {
    run_c<TI, D, 1>(a, s);
  }
  return (int)hipGetLastError();
}

int launch_recurrent(const RecurrentArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == 0) return a.D == 128 ? recurrent_t<bf16, 128>(a, s) : recurrent_t<bf16, 64>(a, s);
  return a.D == 128 ? recurrent_t<float, 128>(a, s) : recurrent_t<float, 64>(a, s);
}

} // namespace gdn
