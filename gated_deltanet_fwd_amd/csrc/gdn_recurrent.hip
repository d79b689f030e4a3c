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
// by moving the states, k_recurrent_run for longer runs, bound by what a token computes.
#include <atomic>
#include <climits>

#include "gdn_step.h"

namespace gdn {

// The wave's place in a grid of (heads x blocks of columns / waves a workgroup, sequences); cb counts
// within a state.
__device__ __forceinline__ bool wave_of(const RecurrentArgs& a, int blocks, int* n, int* h, int* j, int* cb) {
  const int w = (int)(blockIdx.x * (blockDim.x >> 6)) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  *n = (int)(blockIdx.z * MAX_GRID_Y + blockIdx.y);
  *h = w / blocks;
  *cb = w % blocks;
  *j = (int)(((uint64_t)*h * a.g_mul) >> 32);
  return *h < a.HV && *n < a.N;
}

// ------------------------------------------------------------------------------------------------
// One token, or a few: a wave holds COLS = 32 columns, lane (kg, cg) = (lane / 8, lane % 8) the D / 8
// keys from kg D / 8 on of columns 4 cg .. 4 cg + 3, so a load or store covers whole 128-byte lines.
// (COLS = 16, for few waves and several tokens: half the lanes a row, twice the groups of keys, and
// half of the arithmetic a token, which is what a chain of tokens waits for.)
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

template <typename TI, int D, StepKind KIND, int COLS>
__global__ __launch_bounds__(256)
__attribute__((amdgpu_waves_per_eu(KIND == ONE_TOKEN ? 3 : 1, KIND == ONE_TOKEN ? 3 : 8))) void k_recurrent_step(RecurrentArgs a) {
  constexpr int CG = COLS / 4, KPL = D * CG / 64, CB = D / COLS; // lanes a row, keys a lane, waves a state
  typedef typename Vec<TI, KPL>::type kvec;
  const int lane = threadIdx.x & 63, cg = lane % CG, kg = lane / CG;
  int n, h, j, cb; // sequence, value head, q/k head, block of columns
  if (!wave_of(a, CB, &n, &h, &j, &cb)) return;
  cb *= COLS;
  // after the sums over the keys a lane keeps the totals of one column, 2 (lane / 32) + lane / 16 % 2
  // of its four, and the value and output of that column
  const int col = cb + 4 * cg + 2 * (lane >> 5) + ((lane >> 4) & 1);
  const bool writes = !(lane & (16 - CG));
  TI* o = (TI*)a.o + (int64_t)h * D + col;
  const int64_t os = (int64_t)a.HV * D;
  const SeqSpan sp = seq_span(a.cu, a.slot_in, a.slot_out, n, a.T, a.n_slots);
  if (KIND == RUN_OF_TOKENS && sp.t1 - sp.t0 > a.len_max) return;
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
  const auto row_sum = [](float x) { // over the key groups of a row of 16 lanes, in every lane
    if constexpr (COLS == 16) x += dpp<0x124>(x);
    return x + dpp<0x128>(x);
  };
  const auto all = [&](float x) { // sum over the key groups, in every lane
    x = row_sum(x);
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
      s1[c] = row_sum(s1[c]);
      s2[c] = row_sum(s2[c]);
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
// Runs, 16 tokens at a time. With S the state before a block, G_i = a_0 .. a_i, D_ij = a_{j+1} .. a_i
// (products of decays, 1 for i = j, none for i < j) and kh, qh the normalised rows, the recurrence
// unrolls to
//
//   (I + L) U = diag(beta) (V - diag(G) Kh S),   L_ij = beta_i D_ij kh_i.kh_j  (j < i)
//   O = diag(G) Qh S + P U,                      P_ij = D_ij qh_i.kh_j         (j <= i)
//   S <- G_15 S + Kh^T diag(D_15,j) U
//
// in FP32 throughout, the products on v_mfma_f32_16x16x4. A workgroup holds 16 NB columns of a state, 16
// in each of its first NB waves, and takes NB blocks a turn. What does not depend on S (Gram products,
// decays, the inverse T of I + L by forward substitution) the other NB waves prepare in LDS a turn
// ahead, a block each. With NB = 2 every wave has a SIMD to itself, and neither half waits for the
// other's matrix instructions; with NB = 4 half as much is prepared for the same columns. Lane (g, n) =
// (lane / 16, lane % 16) holds rows g D/4 .. of column n of S; with the rows in the order (i, r) ->
// g D/4 + 4 r + i the same registers are the products' B operand and the update's accumulators. A
// product sums over the key rows in any order, so the K and Q rows lie in LDS in the order that makes
// their A operands whole 16-byte reads.
// What bounds it is the matrix unit, and the products' latency one after the other: 104 (D = 128) or 56
// (64) instructions of 32 cycles a block and wave. So with CUs to spare and long runs a workgroup takes
// 16 columns, two waves with half of the rows (r) of each (KS = 2) and four that prepare; the halves add
// up K S through LDS while they multiply Q S, and the second's share of the outputs goes to the first.
// 700 tokens, f32, 64 wide, 8 heads and 5 sequences: 42 us, 60 ns a token; with KS = 1 50 us (49 with
// nothing left to prepare); token by token in the step kernel 680 ns a token.
// What is not finite in a block, be it an input, a product of rising decays or a sum, reaches all of its
// tokens through the zeros above the diagonals (0 inf is NaN), also where the recurrence has ordinary
// numbers: before a NaN, or where the decays rise over an empty state. It goes through U into every row of S
// and never leaves S again. So where the last state is not finite a wave runs its columns of the sequence
// once more from the start, token by token as the step kernel does.
template <typename TI, int D, int NB, int KS>
__global__ __launch_bounds__(128 * NB, 2) void k_recurrent_run(RecurrentArgs a) {
  constexpr int C = 16, DG = D / 4, R = D / 16; // tokens a block, rows a lane, tiles
  constexpr int RH = R / KS, VW = RH < 4 ? RH : 4; // tiles of a wave, floats of an operand read
  constexpr int COLS = KS == 1 ? 16 * NB : 16;     // columns of a workgroup
  constexpr int LD = D + 4, LT = 20;               // LDS row strides
  typedef typename Vec<TI, 8>::type vec8;
  struct alignas(16) Prep { // of one block
    float k[C][LD], q[C][LD]; // rows, permuted
    float t[C][LT], p[C][LT]; // T diag(beta), P
    float gk[C], gq[C], w[C], g_last[C]; // G rk, G rq, D_15,j rk_j, G_15
  };
  typedef float opnd __attribute__((ext_vector_type(VW)));
  extern __shared__ __attribute__((aligned(16))) float lds[];
  Prep* prep = reinterpret_cast<Prep*>(lds); // of two turns
  struct Exchange { // KS = 2
    f32x4 ks[2][2][64], o[2][64]; // each half's K S, of even and odd exchanges; the second half's outputs, of blocks
  };
  Exchange* xch = reinterpret_cast<Exchange*>(prep + 2 * NB);
  int* done = reinterpret_cast<int*>(&prep[0].t[0][C]); // exchanges that each half has made (in padding)
  const int lane = threadIdx.x & 63, g = lane >> 4, n16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // KS = 2: waves 0 and 1 hold the halves, 2, 3, 6 and 7 prepare, 4 and 5 would share the halves' SIMDs
  const bool prepares = KS == 1 ? wave >= NB : (wave & 2) != 0, idle = KS == 2 && (wave & 6) == 4;
  const int wv = KS == 1 ? wave & (NB - 1) : (wave >> 2) * 2 + (wave & 1), kh = KS == 1 ? 0 : wave & 1;
  const int h = blockIdx.x / (D / COLS), j = (int)(((uint64_t)h * a.g_mul) >> 32);
  int n = blockIdx.z * MAX_GRID_Y + blockIdx.y;
  if (n >= a.N) return;
  // the longest sequences first: where the workgroups outnumber the CUs, one of those would end last (12
  // sequences of up to 300 tokens, 48 heads, 128 wide, bf16: 138 us, 146 as they come)
  if (a.N <= 16) n = (int)(a.order >> (4 * n)) & 15;
  const int col = h * D + (blockIdx.x % (D / COLS)) * COLS + (KS == 1 ? wv * 16 : 0) + n16; // in a row of v and o
  const int os = a.HV * D;
  const SeqSpan sp = seq_span(a.cu, a.slot_in, a.slot_out, n, a.T, a.n_slots);
  if (sp.t1 - sp.t0 < a.len_min) return;
  if (!sp.ok) {
    for (int t = sp.t0 + g; t < sp.t1 && !prepares && !idle && kh == 0; t += 4) ((TI*)a.o)[(int64_t)t * os + col] = (TI)__builtin_nanf("");
    return;
  }
  const int64_t hd = (int64_t)a.HV * D * D, head = (int64_t)h * D * D;
  const int at = (g * DG + 4 * kh * RH) * D + (col - h * D);
  f32x4 S[RH];
  // the block at t: lane (g, i) loads token i's rows g D/4 .. of k and q
  struct Rows {
    vec8 k[DG / 8], q[DG / 8];
    float g, beta;
  };
  const auto load = [&](Rows& r, int t) {
    const int tok = min(t + n16, sp.t1 - 1);
    const TI* kp = (const TI*)a.k + (int64_t)tok * a.ks + (j * D + g * DG);
    const TI* qp = (const TI*)a.q + (int64_t)tok * a.qs + (j * D + g * DG);
#pragma unroll
    for (int e = 0; e < DG / 8; ++e) {
      r.k[e] = reinterpret_cast<const vec8*>(kp)[e];
      r.q[e] = reinterpret_cast<const vec8*>(qp)[e];
    }
    r.g = a.g[(int64_t)tok * a.HV + h];
    r.beta = a.beta[(int64_t)tok * a.HV + h];
  };
  // v and o of the block at t, through a buffer that ends with the sequence: tokens past the end load
  // zeros and are not stored, and no branch makes a wait of one block's access cover another's
  const auto rows_at = [&](const TI* p, int t, int64_t stride) {
    const int64_t from = (int64_t)t * stride;
    return make_rsrc(p + from, max(min(sp.t1 - t, C), 0) * (int)stride * (int)sizeof(TI));
  };
  const int lane_v = (4 * g * (int)a.vs + col) * (int)sizeof(TI), lane_o = (4 * g * os + col) * (int)sizeof(TI);
  const auto load_v = [&](float v[4], int t) { // tokens t + 4 g + s of this lane's column
    const __amdgpu_buffer_rsrc_t r = rows_at((const TI*)a.v, min(t, sp.t1), a.vs);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int off = lane_v + s * (int)a.vs * (int)sizeof(TI);
      if constexpr (sizeof(TI) == 2) v[s] = (float)__builtin_bit_cast(bf16, __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
      else v[s] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    }
  };
  const auto all_groups = [](float x) { // sum over g, in every lane
    Pair p = swap16(x, copy_of(x));
    p = swap32(p.x + p.y, copy_of(p.x + p.y));
    return p.x + p.y;
  };
  const auto mfma1 = [](float x, float y, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(x, y, c, 0, 0, 0); };
  const auto prepare = [&](Prep& b, Rows& r, int t) { // r then takes the wave's block of the next turn
    const bool live = t + n16 < sp.t1; // tokens past the end: zero rows, no decay, nothing written
    float kf[DG], qf[DG];
#pragma unroll
    for (int e = 0; e < DG / 8; ++e) {
      unpack<TI, 8>(r.k[e], kf + 8 * e);
      unpack<TI, 8>(r.q[e], qf + 8 * e);
    }
    float kk = 0.f, qq = 0.f;
    f32x4 gram = zero4(), qk = zero4();
#pragma unroll
    for (int m = 0; m < DG; ++m) {
      kf[m] = live ? kf[m] : 0.f;
      qf[m] = live ? qf[m] : 0.f;
      kk = __builtin_fmaf(kf[m], kf[m], kk);
      qq = __builtin_fmaf(qf[m], qf[m], qq);
      gram = mfma1(kf[m], kf[m], gram); // rows i = 4 g + s, column n16
      qk = mfma1(qf[m], kf[m], qk);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < R; x += 4) {
        *reinterpret_cast<f32x4*>(&b.k[n16][g * DG + i * R + x]) =
            f32x4{kf[4 * x + i], kf[4 * x + 4 + i], kf[4 * x + 8 + i], kf[4 * x + 12 + i]};
        *reinterpret_cast<f32x4*>(&b.q[n16][g * DG + i * R + x]) =
            f32x4{qf[4 * x + i], qf[4 * x + 4 + i], qf[4 * x + 8 + i], qf[4 * x + 12 + i]};
      }
    const float al = live ? __expf(r.g) : 1.f, be = live ? r.beta : 0.f;
    // What follows hides the loads. With 64 columns a workgroup the other half is the longer one, and
    // they cost it 3% here (12 sequences of 300 tokens, 48 heads, 128 wide), so they come last.
    if constexpr (NB == 2 || KS == 2) load(r, t + NB * C);
    const float rk = a.l2norm ? inv_sqrt(all_groups(kk) + 1e-6f) : 1.f;
    const float rq = a.l2norm ? inv_sqrt(all_groups(qq) + 1e-6f) : 1.f;
    // running products: G of token n16, and D_ij of this lane's column j = n16
    float gp = 1.f, gi = 1.f, d = 0.f, dij[4];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float ai = lane_value(al, i);
      gp *= ai;
      gi = i == n16 ? gp : gi;
      d = i == n16 ? 1.f : d * ai;
      dij[i & 3] = (i >> 2) == g ? d : dij[i & 3];
    }
    // scale the Gram products; L goes through b.t to be read row by row
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int i = 4 * g + s;
      const float rki = __shfl(rk, i), rqi = __shfl(rq, i), bei = __shfl(be, i);
      b.t[i][n16] = i > n16 ? bei * rki * rk * dij[s] * gram[s] : 0.f;
      b.p[i][n16] = i >= n16 ? rqi * rk * dij[s] * qk[s] : 0.f;
    }
    if (g == 0) {
      b.gk[n16] = gi * rk;
      b.gq[n16] = gi * rq;
      b.w[n16] = d * rk;
      b.g_last[n16] = gp;
    }
    // T = (I + L)^-1, column n16: T_i = e_i - sum_{j < i} L_ij T_j (the wave's own LDS writes above
    // are in order with these reads)
    __builtin_amdgcn_wave_barrier();
    float T[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float x = i == n16 ? 1.f : 0.f;
#pragma unroll
      for (int q4 = 0; q4 < (i + 3) / 4; ++q4) {
        const f32x4 l = *reinterpret_cast<const f32x4*>(&b.t[i][4 * q4]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * q4 + e < i) x = __builtin_fmaf(-l[e], T[4 * q4 + e], x);
      }
      T[i] = x;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < C; ++i)
      if ((i >> 2) == g) b.t[i][n16] = T[i] * be;
    if constexpr (NB > 2 && KS == 1) load(r, t + NB * C);
  };
  // The operands of the products with S, read while the block before is finished: the waits for LDS
  // would otherwise stand between the products.
  opnd ka[4][RH / VW], qa[4][RH / VW];
  const auto operands = [&](const Prep& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < RH / VW; ++x) {
        ka[i][x] = *reinterpret_cast<const opnd*>(&b.k[n16][g * DG + i * R + kh * RH + VW * x]);
        qa[i][x] = *reinterpret_cast<const opnd*>(&b.q[n16][g * DG + i * R + kh * RH + VW * x]);
      }
  };
  const auto store_o = [&](const f32x4& x4, int t) {
    const __amdgpu_buffer_rsrc_t to = rows_at((const TI*)a.o, t, os);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int off = lane_o + s * os * (int)sizeof(TI);
      const TI x = (TI)x4[s];
      if constexpr (sizeof(TI) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, x), to, off, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, x), to, off, 0, 0);
    }
  };
  // The halves' exchange: a half writes its part, then counts the exchange; the other reads the count, then
  // the part. Parts of even and odd exchanges have places of their own: one is written again two exchanges
  // later, and by then the other half has counted one after reading it. Both halves go through the same
  // blocks (an exchange each), agree at the end, and go through the same tokens if they run again, so the
  // wait ends.
  const auto lds_order = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local"); };
  const auto others_count = [&] {
    return __builtin_amdgcn_readfirstlane(__hip_atomic_load(done + 1 - kh, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP));
  };
  const auto count = [&](int exchanges) {
    lds_order();
    __hip_atomic_store(done + kh, exchanges, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  };
  const auto wait_for = [&](int exchanges) {
    while (others_count() < exchanges) {}
    lds_order();
  };
  f32x4 o; // KS = 2: between the blocks, the first half's part of the outputs of the one before
  // block i of the sequence, at token t
  const auto block = [&](int i, const float v[4], int t) {
    const Prep& b = prep[i % (2 * NB)];
    const f32x4 gk = *reinterpret_cast<const f32x4*>(&b.gk[4 * g]), gq = *reinterpret_cast<const f32x4*>(&b.gq[4 * g]);
    const f32x4 w = *reinterpret_cast<const f32x4*>(&b.w[4 * g]);
    const f32x4 ta = *reinterpret_cast<const f32x4*>(&b.t[n16][4 * g]), pa = *reinterpret_cast<const f32x4*>(&b.p[n16][4 * g]);
    const float last = b.g_last[0];
    // the update's: lane (g, 4 y + i): rows y D/4 + 4 r + i of token 4 g + s
    opnd ua[4][RH / VW];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int x = 0; x < RH / VW; ++x)
        ua[s][x] = *reinterpret_cast<const opnd*>(&b.k[4 * g + s][(n16 >> 2) * DG + (n16 & 3) * R + kh * RH + VW * x]);
    __builtin_amdgcn_sched_barrier(0);
    f32x4 ks = zero4(), qs = zero4(), other;
    int seen = 0;
    if constexpr (KS == 1) {
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          ks = mfma1(ka[y][r / VW][r % VW], S[r][y], ks);
          qs = mfma1(qa[y][r / VW][r % VW], S[r][y], qs);
        }
    } else {
      f32x4 ks2 = zero4(), qs2 = zero4();
#pragma unroll
      for (int y = 0; y < 4; y += 2)
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          ks = mfma1(ka[y][0][r], S[r][y], ks);
          ks2 = mfma1(ka[y + 1][0][r], S[r][y + 1], ks2);
        }
      __builtin_amdgcn_sched_barrier(0);
      const auto q_part = [&](int y) {
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          f32x4& to = r & 1 ? qs2 : qs;
          to = mfma1(qa[y][0][r], S[r][y], to);
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      q_part(0);
      ks += ks2;
      xch->ks[i & 1][kh][lane] = ks;
      count(i + 1);
      __builtin_amdgcn_sched_barrier(0);
      q_part(1);
      q_part(2);
      seen = others_count();
      lds_order();
      other = xch->ks[i & 1][1 - kh][lane];
      __builtin_amdgcn_sched_barrier(0);
      q_part(3);
      qs += qs2;
    }
    __builtin_amdgcn_sched_barrier(0);
    if (t + C < sp.t1) {
      if (i % NB == NB - 1) __syncthreads(); // the next turn is ready; of this one everything is in registers
      if constexpr (KS == 1) operands(prep[(i + 1) % (2 * NB)]);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (KS == 2) {
      if (seen <= i) {
        wait_for(i + 1);
        other = xch->ks[i & 1][1 - kh][lane];
      }
      ks += other;
      if (kh == 0 && i > 0) store_o(o + xch->o[(i - 1) & 1][lane], t - C);
    }
    f32x4 rhs, u = zero4(), u2 = zero4();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      rhs[s] = __builtin_fmaf(-gk[s], ks[s], v[s]);
      o[s] = gq[s] * qs[s];
    }
    u = mfma1(ta[0], rhs[0], u);
    u2 = mfma1(ta[1], rhs[1], u2);
    u = mfma1(ta[2], rhs[2], u);
    u2 = mfma1(ta[3], rhs[3], u2);
    if constexpr (KS == 2) operands(prep[(i + 1) % (2 * NB)]); // of no use after the last block
#pragma unroll
    for (int r = 0; r < RH; ++r) S[r] *= last;
    u += u2;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float wu = w[s] * u[s]; // of token 4 g + s
#pragma unroll
      for (int r = 0; r < RH; ++r) S[r] = mfma1(ua[s][r / VW][r % VW], wu, S[r]);
    }
    if (KS == 1 || kh == 1) {
#pragma unroll
      for (int s = 0; s < 4; ++s) o = mfma1(pa[s], u[s], o);
    }
    if constexpr (KS == 1) store_o(o, t);
    else if (kh == 1) xch->o[i & 1][lane] = o;
  };
  if (idle) {
    for (int t = sp.t0; t < sp.t1; t += NB * C) __syncthreads();
    return;
  }
  if (prepares) {
    if (sp.t0 >= sp.t1) return;
    Rows r;
    load(r, sp.t0 + wv * C);
    int buf = 0;
    for (int t = sp.t0; t < sp.t1; t += NB * C, buf ^= NB) {
      if (t + wv * C < sp.t1) prepare(prep[buf + wv], r, t + wv * C);
      __syncthreads(); // this turn is ready, and the one before it has been used
    }
    return;
  }
  const auto load_state = [&] {
    const float* p = a.states + (sp.in < 0 ? 0 : sp.in) * hd + head + at;
#pragma unroll
    for (int r = 0; r < RH; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[r][i] = keepf(p[(4 * r + i) * D], sp.in >= 0);
  };
  load_state();
  if (sp.t0 < sp.t1) {
    float v0[4], v1[4];
    load_v(v0, sp.t0);
    if constexpr (KS == 2) done[kh] = 0; // seen by the other half after the barrier
    __syncthreads(); // the first turn is ready
    operands(prep[0]);
    int i = 0;
#pragma unroll 1
    for (int t = sp.t0; t < sp.t1; t += 2 * C, i += 2) {
      load_v(v1, t + C);
      block(i, v0, t);
      if (t + C >= sp.t1) break;
      load_v(v0, t + 2 * C);
      block(i + 1, v1, t + C);
    }
    float sum = 0.f; // of 0 s over the state's values s: NaN if one is not finite
#pragma unroll
    for (int r = 0; r < RH; ++r)
#pragma unroll
      for (int y = 0; y < 4; ++y) sum = __builtin_fmaf(0.f, S[r][y], sum);
    bool finite = __ballot(sum != sum) == 0;
    int x = 0; // KS = 2: exchanges made
    if constexpr (KS == 2) { // the halves agree
      x = (sp.t1 - sp.t0 + C - 1) / C; // one a block
      xch->ks[x & 1][kh][lane] = f32x4{finite ? 0.f : 1.f, 0.f, 0.f, 0.f};
      count(++x);
      wait_for(x);
      finite = finite && xch->ks[(x - 1) & 1][1 - kh][lane][0] == 0.f;
      if (kh == 0) store_o(o + xch->o[x & 1][lane], sp.t0 + (x - 2) * C); // of the last block, x - 2
    }
    if (__builtin_expect(!finite, 0)) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent"); // the outputs so far are written before they are again
      load_state();
#pragma unroll 1
      for (int t = sp.t0; t < sp.t1; ++t) {
        const TI* kp = (const TI*)a.k + (int64_t)t * a.ks + (j * D + g * DG);
        const TI* qp = (const TI*)a.q + (int64_t)t * a.qs + (j * D + g * DG);
        float kk = 0.f, qq = 0.f, qk = 0.f, s1 = 0.f, s2 = 0.f, k[RH][4];
#pragma unroll 1
        for (int m = 0; m < DG; ++m) {
          const float km = (float)kp[m], qm = (float)qp[m];
          kk = __builtin_fmaf(km, km, kk);
          qq = __builtin_fmaf(qm, qm, qq);
          qk = __builtin_fmaf(qm, km, qk);
        }
#pragma unroll
        for (int r = 0; r < RH; ++r)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            k[r][y] = (float)kp[4 * (kh * RH + r) + y];
            s1 = __builtin_fmaf(S[r][y], k[r][y], s1);
            s2 = __builtin_fmaf(S[r][y], (float)qp[4 * (kh * RH + r) + y], s2);
          }
        s1 = all_groups(s1);
        s2 = all_groups(s2);
        if constexpr (KS == 2) {
          xch->ks[x & 1][kh][lane] = f32x4{s1, s2, 0.f, 0.f};
          count(++x);
          wait_for(x);
          const f32x4 other = xch->ks[(x - 1) & 1][1 - kh][lane];
          s1 += other[0];
          s2 += other[1];
        }
        const float rk = a.l2norm ? inv_sqrt(all_groups(kk) + 1e-6f) : 1.f;
        const float rq = a.l2norm ? inv_sqrt(all_groups(qq) + 1e-6f) : 1.f;
        const float al = __expf(a.g[(int64_t)t * a.HV + h]);
        const float u = a.beta[(int64_t)t * a.HV + h] * rk * __builtin_fmaf(-al * rk, s1, (float)((const TI*)a.v)[(int64_t)t * a.vs + col]);
        const float out = rq * __builtin_fmaf(al, s2, all_groups(qk) * u);
        if (g == 0 && kh == 0) ((TI*)a.o)[(int64_t)t * os + col] = (TI)out;
#pragma unroll
        for (int r = 0; r < RH; ++r)
#pragma unroll
          for (int y = 0; y < 4; ++y) S[r][y] = __builtin_fmaf(k[r][y], u, al * S[r][y]);
      }
    }
  }
  if (sp.out >= 0) {
    float* p = a.states + sp.out * hd + head + at;
#pragma unroll
    for (int r = 0; r < RH; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) p[(4 * r + i) * D] = S[r][i];
  }
}
// LDS of a workgroup: the rows, T, P and factors of two turns of NB blocks, and what the halves exchange
// (D = 128, KS = 2: all of the 160 KiB)
constexpr unsigned run_lds(int D, int NB, int KS) {
  return 2 * NB * 4 * (2 * 16 * (D + 4) + 2 * 16 * 20 + 4 * 16) + (KS == 2 ? 6 * 1024 : 0);
}

static dim3 grid_of(const RecurrentArgs& a, int x) {
  const unsigned n = (unsigned)a.N;
  return dim3((unsigned)x, n < MAX_GRID_Y ? n : MAX_GRID_Y, (n + MAX_GRID_Y - 1) / MAX_GRID_Y);
}

template <typename TI, int D, int NB, int KS>
static int run_t(const RecurrentArgs& a, hipStream_t s) {
  constexpr unsigned lds = run_lds(D, NB, KS);
  if constexpr (lds > 64 * 1024) { // more than the runtime gives unasked: asked for once on each device
    static std::atomic<uint64_t> asked{0};
    int dev = 0;
    if (const hipError_t e = hipGetDevice(&dev)) return (int)e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!(asked.load(std::memory_order_relaxed) & bit)) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_recurrent_run<TI, D, NB, KS>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return (int)e;
      asked.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL((k_recurrent_run<TI, D, NB, KS>), grid_of(a, a.HV * (KS == 1 ? D / (16 * NB) : D / 16)), dim3(128 * NB), lds, s, a);
  return (int)hipGetLastError();
}

// The step kernel, its columns a wave and waves a workgroup by the number of waves of 32 columns. With
// few, a wave to a workgroup spreads them over more CUs, so that their stores do not queue at one (us in
// workgroups of 4 / 1, 128 wide, bf16, one token: 1152 waves 8.0 / 6.8, 3072 19.0 / 21.1). With fewer
// still, and several tokens, 16 columns (us with 32 / 16, 6 kept tokens: 192 waves 10.1 / 9.6, 576 13.6 /
// 16.1).
template <typename TI, int D, StepKind KIND>
static int step_t(const RecurrentArgs& a, hipStream_t s) {
  constexpr int64_t SPREAD = 1280, HALVED = 384;
  const int64_t waves = (int64_t)a.live * a.HV * (D / 32);
  if (KIND != ONE_TOKEN && a.longest > 1 && waves <= HALVED) {
    constexpr int GROUP = KIND == KEEP_EACH ? 1 : 4, COLS = KIND == ONE_TOKEN ? 32 : 16;
    hipLaunchKernelGGL((k_recurrent_step<TI, D, KIND, COLS>), grid_of(a, (a.HV * (D / COLS) + GROUP - 1) / GROUP),
                       dim3(64 * GROUP), 0, s, a);
  } else {
    const int group = waves <= SPREAD ? 1 : 4;
    hipLaunchKernelGGL((k_recurrent_step<TI, D, KIND, 32>), grid_of(a, (a.HV * (D / 32) + group - 1) / group),
                       dim3(64 * group), group == 1 ? 0 : STEP_LDS, s, a);
  }
  return (int)hipGetLastError();
}

// The kernel by the host's lengths. A run's workgroup pays for whole blocks of 16 tokens and for the start
// of its two halves, so it gains from 7 tokens on, and with more workgroups than CUs later (us step / run,
// 48 heads, 128 wide, bf16: 1 sequence of 4 tokens 6.2 / 7.6, of 8 9.0 / 7.8; 32 sequences of 12 71 / 84, of
// 24 118 / 112). 32 columns a workgroup while each then has a CU, 64 beyond (us with 32 / 64, of 256 tokens:
// 1 sequence 35 / 43, 2 61 / 47). Two waves a column while each 16 columns have a CU and the run is long
// enough to pay for the start (us with two / one, 8 heads: 64 tokens 12.9 / 12.9, 256 27 / 34). With slot_tok
// every token's state is wanted: always the step.
// Beside longer sequences, short ones go to a step launch of their own when they alone would fill the CUs
// several times with run workgroups, each of which prepares 16 tokens for a few. Each kernel leaves the
// other's sequences by their length on the device. (us apart / in one run launch, 48 heads: 255 sequences of
// 1 token and one of 13 327 / 664, 16 of 6 and one of 100 47 / 67, 12 of 6 and one of 300 64 / 58; of 12
// tokens, not taken as short, 24 and one of 300 123 / 113.)
template <typename TI, int D>
static int recurrent_t(RecurrentArgs a, hipStream_t s) {
  constexpr int CUS = 256, SPLIT = 6;
  a.len_min = INT_MIN;
  a.len_max = INT_MAX;
  if (a.slot_tok) return step_t<TI, D, KEEP_EACH>(a, s);
  if (!a.cu) return step_t<TI, D, ONE_TOKEN>(a, s);
  const auto groups = [&](int n) { return (int64_t)n * a.HV * (D / 64); };
  if (a.longest <= (groups(a.live) <= CUS ? 6 : 12)) return step_t<TI, D, RUN_OF_TOKENS>(a, s);
  if (a.longs > 0 && groups(a.N - a.longs) > SPLIT * CUS) {
    RecurrentArgs b = a;
    b.len_max = b.longest = SHORT_RUN;
    b.live = a.live - a.longs;
    if (const int e = step_t<TI, D, RUN_OF_TOKENS>(b, s)) return e;
    a.len_min = SHORT_RUN + 1;
    a.live = a.longs;
  }
  const int64_t run_groups = groups(a.live);
  if (4 * run_groups <= CUS && a.longest > 64) return run_t<TI, D, 4, 2>(a, s);
  return 2 * run_groups <= CUS ? run_t<TI, D, 2, 1>(a, s) : run_t<TI, D, 4, 1>(a, s);
}

int launch_recurrent(const RecurrentArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == 0) return a.D == 128 ? recurrent_t<bf16, 128>(a, s) : recurrent_t<bf16, 64>(a, s);
  return a.D == 128 ? recurrent_t<float, 128>(a, s) : recurrent_t<float, 64>(a, s);
}

} // namespace gdn
