// What a serving step reads, made from the requests' lengths (gfx950): sequence starts, positions, block tables and
// slots. Integers and a few kilobytes: it costs its latency, a chain of a few memory accesses and barriers. The whole
// of it depends on two running sums over the requests (tokens, new blocks), which every workgroup makes for itself
// in LDS, at once with the others, rather than wait for one that makes them for all. 256 requests of one token 3.6 us,
// of 64 tokens 3.8 (in a graph).
#include <algorithm>

#include "gdn_device.h"

namespace gdn {

constexpr int MAPS_SEQS = 4096;

// x + y, at most 2^31 - 1 (for x and y at most that): sums of lengths that nobody can have stay too large to fit
__device__ __forceinline__ unsigned add_up_to(unsigned x, unsigned y) { return min(x + y, 0x7fffffffu); }
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned scan_step(unsigned x) {
  return add_up_to(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false));
}
// Inclusive sums over a wave's lanes (steps as in wave_prefix_sum)
__device__ __forceinline__ unsigned wave_sums(unsigned x) {
  x = scan_step<0x111, 0xf>(x);
  x = scan_step<0x112, 0xf>(x);
  x = scan_step<0x114, 0xf>(x);
  x = scan_step<0x118, 0xf>(x);
  x = scan_step<0x142, 0xa>(x);
  return scan_step<0x143, 0xc>(x);
}

// Every workgroup fills tokens and the new entries of the table; workgroup 0 also writes what is one value a
// request, after all of its inputs are read.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void k_maps(MapsArgs a) {
  constexpr int WAVES = THREADS / 64;
  __shared__ int ends[MAPS_SEQS], shift[MAPS_SEQS], taken[MAPS_SEQS]; // tokens so far, position - token, blocks before
  __shared__ uint2 sums[WAVES], fitting[WAVES]; // a wave's sums; the sums up to its last request that fits
  const int B = a.block, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool update = blockIdx.x == 0;
  const unsigned count = min(max(a.free_count[0], 0), a.n_free);
  const int64_t room = (int64_t)a.max_blocks * B < 0x7fffffff ? (int64_t)a.max_blocks * B : 0x7fffffff; // of a request
  const auto full = [&](int x) { return (int)(((uint64_t)(unsigned)x * a.block_mul) >> a.block_shift); }; // x / B
  const auto blocks = [&](int x) { return x == 0 ? 0 : full(x - 1) + 1; };
  uint2 carry = {0, 0}, total = {0, 0}; // sums over all requests so far, over those that fit (tokens, blocks)
  for (int r0 = 0; r0 < a.N; r0 += THREADS) {
    const int r = r0 + (int)threadIdx.x;
    int len = 0, ctx = 0, given = 0, in = -1;
    bool fine = false;
    const int32_t* row = a.table;
    if (r < a.N) {
      len = a.lengths[r];
      given = ctx = a.contexts[r];
      row += (int64_t)r * a.max_blocks;
      fine = ctx >= 0 && ctx <= room;
      if (!fine) ctx = 0;
      if (!fine || len < 0 || ctx + (int64_t)len > room) len = 0;
      if (update && ctx > 0) in = row[full(ctx - 1)];
    }
    const int held = blocks(ctx), need = blocks(ctx + len) - held;
    uint2 s = {wave_sums((unsigned)len), wave_sums((unsigned)need)};
    if (lane == 63) sums[wave] = s;
    __syncthreads();
    uint2 before = carry;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const uint2 x = sums[w];
      carry.x = add_up_to(carry.x, x.x);
      carry.y = add_up_to(carry.y, x.y);
      if (w + 1 == wave) before = carry;
    }
    s.x = add_up_to(s.x, before.x);
    s.y = add_up_to(s.y, before.y);
    const bool fits = s.x <= (unsigned)a.T && s.y <= count; // sums rise, so those that fit are the first ones
    const uint64_t which = __ballot(fits);
    if (which == 0 ? lane == 0 : lane == 63 - __builtin_clzll(which)) fitting[wave] = which ? s : uint2{0, 0};
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const uint2 x = fitting[w];
      total.x = max(total.x, x.x);
      total.y = max(total.y, x.y);
    }
    if (r < a.N) {
      if (!fits) len = 0;
      const int end = (int)(fits ? s.x : total.x), first = (int)(fits ? s.y - need : total.y);
      ends[r] = end;
      shift[r] = ctx - (end - len);
      taken[r] = first;
      if (update) {
        int out = in; // a new token's block that the request has already is its last one
        if (len > 0) {
          const int b = full(ctx + len - 1);
          if (b >= held) out = a.free_list[count - 1 - (first + b - held)];
        }
        if (a.cu) a.cu[r + 1] = end;
        if (a.granted) a.granted[r] = len;
        if (a.slot_in) a.slot_in[r] = in;
        if (a.slot_out) a.slot_out[r] = out;
        if (a.contexts_out) a.contexts_out[r] = fine ? ctx + len : given;
      }
    }
  }
  if (update && threadIdx.x == 0) {
    if (a.cu) a.cu[0] = 0;
    if (a.free_count_out) a.free_count_out[0] = (int)(count - total.y);
  }
  if (!a.fill) return;
  __syncthreads();
  for (int64_t t = (int64_t)blockIdx.x * THREADS + threadIdx.x; t < a.T; t += (int64_t)gridDim.x * THREADS) {
    int pos = 0, keep = -1;
    int64_t slot = -1;
    if (t < total.x) {
      int lo = 0, hi = a.N - 1; // the first request that ends behind t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > t) hi = mid;
        else lo = mid + 1;
      }
      const int begin = lo > 0 ? ends[lo - 1] : 0;
      pos = (int)t + shift[lo];
      const int b = full(pos), at = pos - b * B, held = blocks(begin + shift[lo]);
      int32_t* entry = a.table + (int64_t)lo * a.max_blocks + b;
      int id;
      if (b < held) id = *entry;
      else {
        id = a.free_list[count - 1 - (taken[lo] + b - held)];
        if (at == 0) *entry = id; // the token that enters a block
      }
      slot = (int64_t)id * B + at;
      if (at == B - 1 && t + 1 < ends[lo]) keep = id;
    }
    if (a.positions) a.positions[t] = pos;
    if (a.token_slots) a.token_slots[t] = slot;
    if (a.slot_tok) a.slot_tok[t] = keep;
  }
}

// A workgroup for every THREADS tokens. Every one sums over all requests, at the price of its barriers' waves: 256 threads
// up to 512 requests, 1024 for more (us: 256 requests, 16,384 tokens 3.8 and 5.1; 512, 4096 tokens 4.5 and 5.0;
// 4096 requests 17.8 and 13.7).
template <int THREADS>
static int maps_t(const MapsArgs& a, int groups, hipStream_t s) {
  hipLaunchKernelGGL(k_maps<THREADS>, dim3((unsigned)groups), dim3(THREADS), 0, s, a);
  return (int)hipGetLastError();
}
static int maps_any(const MapsArgs& a, int tokens, hipStream_t s) { // for `tokens` tokens a workgroup each of its threads'
  const int most = 1024;
  if (a.N <= 512) return maps_t<256>(a, std::max(1, std::min(most, (int)(((int64_t)tokens + 255) / 256))), s);
  return maps_t<1024>(a, std::max(1, std::min(most, (int)(((int64_t)tokens + 1023) / 1024))), s);
}

// Contexts and the count that move on in place may still be read by another workgroup, so few tokens are left to one
// workgroup, and for more they wait for a launch of their own (us, alone and so: 256 requests, 1024 tokens 5.0 and 7.1; 64,
// 2048 tokens 5.9 and 6.4; 512, 4096 tokens 8.5 and 7.2; 4096 requests and tokens 17.9 and 23.2, another 1.1 alone for each
// 1024 tokens). Alone with 256 threads up to 512 tokens (64 requests: 4.2 us, with 1024 threads 4.6; 2048 tokens 9.3, 5.9).
int launch_maps(const MapsArgs& a0, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  MapsArgs a = a0;
  a.fill = 1;
  if (a.contexts_out != a.contexts && a.free_count_out != a.free_count) return maps_any(a, a.T, s);
  if (a.T <= (a.N <= 512 ? 2048 : 8192)) return a.T <= 512 ? maps_any(a, 1, s) : maps_t<1024>(a, 1, s);
  MapsArgs rest = a;
  a.contexts_out = a.free_count_out = nullptr;
  rest.cu = rest.granted = rest.slot_in = rest.slot_out = nullptr;
  rest.fill = 0;
  if (const int e = maps_any(a, a.T, s)) return e;
  return maps_any(rest, 1, s);
}

} // namespace gdn
