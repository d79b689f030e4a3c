// Linear attention with a decay for each head, recurrent, on cached FP32 states (gfx950): one token a sequence
// when decoding, short runs when drafted tokens are checked or a prompt is extended. Per token and value head
//
//   S = exp(g) S + k v^T,  o = scale S^T q
//
// A wave holds COLS columns of one head's state (a column is a value index; they never mix) in registers from the first
// token to the last, as k_recurrent_step does. It costs moving the states: 256 sequences of 48 heads, 128 wide, one
// token each, 1.61 GB in 266 us (6.05 TB/s; two workgroups a CU, held apart by LDS, 294 us). States are read and written
// non-temporally, and a row leaves as soon as it is made (nothing of a new state waits for a sum). Absent states are
// buffers of no bytes.
#include "gdn_step.h"

namespace gdn {

template <typename TI, int D, bool ONE, bool KEEP, int COLS> // one token a sequence; with slot_tok
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(ONE ? 3 : 1, ONE ? 3 : 8))) void k_linear_step(LinearStepArgs a) {
  constexpr int CG = COLS / 4, KPL = D * CG / 64, CB = D / COLS; // lanes a row, keys a lane, waves a state
  typedef typename Vec<TI, KPL>::type kvec;
  typedef typename Vec<TI, 4>::type vvec;
  const int lane = threadIdx.x & 63, cg = lane % CG, kg = lane / CG;
  const int w = (int)(blockIdx.x * (blockDim.x >> 6)) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = (int)(blockIdx.z * MAX_GRID_Y + blockIdx.y), h = w / CB, cb = w % CB * COLS;
  if (h >= a.HV || n >= a.N) return;
  const int j = (int)(((uint64_t)h * a.g_mul) >> 32);
  const int at4 = cb + 4 * cg; // this lane's four columns
  // after the sum over the keys a lane has the total of one of them
  const int col = at4 + 2 * (lane >> 5) + ((lane >> 4) & 1);
  const bool writes = !(lane & (16 - CG));
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
  const int at = 4 * (kg * KPL * D + at4); // bytes
  const auto state = [&](int slot) {
    return make_rsrc(a.states + (slot < 0 ? 0 : slot) * hd + head, slot < 0 ? 0 : D * D * 4);
  };
  f32x4 S[KPL];
  const __amdgpu_buffer_rsrc_t from = state(sp.in);
#pragma unroll
  for (int i = 0; i < KPL; ++i)
    S[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, at + 4 * D * i, 0, NT));
  const auto store_row = [&](const __amdgpu_buffer_rsrc_t& to, int i) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4_t, S[i]), to, at + 4 * D * i, 0, KEEP ? WRITE_THROUGH : NT);
  };
  struct Rows {
    kvec k, q;
    vvec v;
    float g;
    int st;
  };
  const TI* qp = (const TI*)a.q + (int64_t)j * D + kg * KPL;
  const TI* kp = (const TI*)a.k + (int64_t)j * D + kg * KPL;
  const TI* vp = (const TI*)a.v + (int64_t)h * D + at4;
  const auto load = [&](Rows& r, int t) {
    r.k = *reinterpret_cast<const kvec*>(kp + t * a.ks);
    r.q = *reinterpret_cast<const kvec*>(qp + t * a.qs);
    r.v = *reinterpret_cast<const vvec*>(vp + t * a.vs);
    r.g = a.g[(int64_t)t * a.gs + h];
    if constexpr (KEEP) r.st = a.slot_tok[t];
  };
  const auto row_sum = [](float x) { // over the key groups of a row of 16 lanes, in every lane
    if constexpr (COLS == 16) x += dpp<0x124>(x);
    return x + dpp<0x128>(x);
  };
  const auto compute = [&](const Rows& r, int t) {
    float kf[KPL], qf[KPL];
    unpack<TI, KPL>(r.k, kf);
    unpack<TI, KPL>(r.q, qf);
    const float al = __expf(r.g);
    int keep = -1;
    bool bad = false;
    if constexpr (ONE && !KEEP) keep = sp.out;
    if constexpr (KEEP) {
      bad = r.st < -1 || r.st >= a.n_slots;
      keep = bad ? -1 : r.st;
    }
    const __amdgpu_buffer_rsrc_t to = state(keep);
    f32x4 s = zero4();
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        S[i][c] = __builtin_fmaf(kf[i], (float)r.v[c], al * S[i][c]);
        s[c] = __builtin_fmaf(S[i][c], qf[i], s[c]);
      }
      if constexpr (ONE || KEEP) {
        store_row(to, i);
        __builtin_amdgcn_sched_barrier(0); // each row leaves as it is made
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) s[c] = row_sum(s[c]);
    Pair x0 = swap32(s[0], s[2]), x1 = swap32(s[1], s[3]);
    x0 = swap16(x0.x + x0.y, x1.x + x1.y);
    const float out = a.scale * (x0.x + x0.y);
    if (writes) o[t * os] = (TI)(bad ? nan : out);
  };
  if constexpr (ONE) {
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

// Waves a workgroup and columns a wave by the number of waves of 32 columns (us, states from memory, 48 heads, 128 wide).
// One wave a workgroup spreads few over all CUs, four keep a CU's waves on neighbouring columns: one token, 192 waves 3.5
// and 4.5, 1152 waves 9.2 and 10.3, 2112 waves 15.0 and 15.5, 12,288 waves 74.5 and 67.6, 49,152 waves 301 and 267. Half the
// columns halve a token's chain where there are several and few waves: four tokens, 16 waves 4.3 and 4.8, 256 waves
// 5.9 either way (states in cache 5.1 and 5.5), 768 waves 8.6 and 8.2.
template <typename TI, int D, bool ONE, bool KEEP>
static int linear_step_t(const LinearStepArgs& a, hipStream_t s) {
  constexpr int64_t SPREAD = 1280, HALVED = 384;
  const int64_t waves = (int64_t)a.live * a.HV * (D / 32);
  const unsigned n = (unsigned)a.N;
  const auto grid = [&](int x) { return dim3((unsigned)x, n < MAX_GRID_Y ? n : MAX_GRID_Y, (n + MAX_GRID_Y - 1) / MAX_GRID_Y); };
  if (!ONE && a.longest > 1 && waves <= HALVED) {
    constexpr int GROUP = KEEP ? 1 : 4, COLS = ONE ? 32 : 16;
    hipLaunchKernelGGL((k_linear_step<TI, D, ONE, KEEP, COLS>), grid((a.HV * (D / COLS) + GROUP - 1) / GROUP), dim3(64 * GROUP), 0, s, a);
  } else {
    const int group = waves <= SPREAD ? 1 : 4;
    hipLaunchKernelGGL((k_linear_step<TI, D, ONE, KEEP, 32>), grid((a.HV * (D / 32) + group - 1) / group), dim3(64 * group), 0, s, a);
  }
  return (int)hipGetLastError();
}
template <typename TI, int D>
static int linear_step_td(const LinearStepArgs& a, hipStream_t s) {
  if (a.slot_tok) return linear_step_t<TI, D, false, true>(a, s);
  return a.cu ? linear_step_t<TI, D, false, false>(a, s) : linear_step_t<TI, D, true, false>(a, s);
}

int launch_linear_step(const LinearStepArgs& a, int dtype, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == 0) return a.D == 128 ? linear_step_td<bf16, 128>(a, s) : linear_step_td<bf16, 64>(a, s);
  return a.D == 128 ? linear_step_td<float, 128>(a, s) : linear_step_td<float, 64>(a, s);
}

} // namespace gdn
