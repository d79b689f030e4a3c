// What a serving step reads, made from the requests' lengths (gfx950): sequence starts, positions, block tables and
// slots. Integers and a few kilobytes: it costs its latency. The whole of it depends on two running sums over the
// requests (tokens, new blocks), which every workgroup makes for itself in LDS, at once with the others, rather
// than wait for one that makes them for all.
#include "gdn_device.h"

namespace gdn {

constexpr int MAPS_THREADS = 1024, MAPS_SEQS = 4096;

// Inclusive sums over the workgroup's threads of two values.
struct Two {
  int64_t x, y;
};
__device__ __forceinline__ Two block_scan(Two v, Two* tmp) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int by = 1; by < 64; by *= 2) {
    const int64_t x = __shfl_up((long long)v.x, by), y = __shfl_up((long long)v.y, by);
    if (lane >= by) {
      v.x += x;
      v.y += y;
    }
  }
  __syncthreads();
  if (lane == 63) tmp[wave] = v;
  __syncthreads();
  for (int i = 0; i < wave; ++i) {
    v.x += tmp[i].x;
    v.y += tmp[i].y;
  }
  return v;
}

// FILL: tokens and the new entries of the table, by all workgroups. UPDATE: what is one value a request, and the
// buffers that may be the inputs' own, by one workgroup that has read all of its inputs before.
template <bool FILL, bool UPDATE>
__global__ __launch_bounds__(MAPS_THREADS) void k_maps(MapsArgs a) {
  __shared__ int ends[MAPS_SEQS], shift[MAPS_SEQS], taken[MAPS_SEQS]; // tokens so far, position - token, blocks before
  __shared__ Two tmp[MAPS_THREADS / 64];
  __shared__ long long most;
  const int B = a.block, count = min(max(a.free_count[0], 0), a.n_free);
  const auto blocks = [&](int64_t upto) { return (int)((upto + B - 1) / B); };
  Two carry = {0, 0};
  int64_t total = 0; // tokens of the requests that fit
  int used = 0;      // blocks they take
  for (int r0 = 0; r0 < a.N; r0 += MAPS_THREADS) {
    const int r = r0 + threadIdx.x;
    int64_t len = 0, ctx = 0;
    int need = 0;
    bool fine = false;
    if (r < a.N) {
      len = a.lengths[r];
      ctx = a.contexts[r];
      fine = ctx >= 0 && ctx <= (int64_t)a.max_blocks * B;
      if (!fine) ctx = 0;
      if (!fine || len < 0 || ctx + len > (int64_t)a.max_blocks * B || ctx + len > 0x7fffffff) len = 0;
      need = blocks(ctx + len) - blocks(ctx);
    }
    Two s = block_scan({len, need}, tmp);
    s.x += carry.x;
    s.y += carry.y;
    const bool fits = s.x <= a.T && s.y <= count;
    // sums rise, so those that fit are the first ones
    __syncthreads();
    if (threadIdx.x == 0) most = total | ((long long)used << 32);
    if (threadIdx.x == MAPS_THREADS - 1) tmp[0] = s;
    __syncthreads();
    if (fits) atomicMax(&most, (long long)(s.x | (s.y << 32)));
    __syncthreads();
    carry = tmp[0];
    total = most & 0x7fffffff;
    used = (int)(most >> 32);
    if (r < a.N) {
      if (!fits) len = 0;
      const int64_t end = fits ? s.x : total, start = end - len;
      const int before = (int)(fits ? s.y - need : used);
      ends[r] = (int)end;
      shift[r] = (int)(ctx - start);
      taken[r] = before;
      if constexpr (UPDATE) {
        const int32_t* row = a.table + (int64_t)r * a.max_blocks;
        const int held = blocks(ctx);
        const int in = ctx > 0 ? row[(ctx - 1) / B] : -1;
        int out = in;
        if (len > 0) {
          const int b = (int)((ctx + len - 1) / B);
          out = b < held ? row[b] : a.free_list[count - 1 - (before + b - held)];
        }
        if (a.cu) a.cu[r + 1] = (int)end;
        if (a.granted) a.granted[r] = (int)len;
        if (a.slot_in) a.slot_in[r] = in;
        if (a.slot_out) a.slot_out[r] = out;
        if (fine && a.contexts_out) a.contexts_out[r] = (int)(ctx + len);
        else if (a.contexts_out && a.contexts_out != a.contexts) a.contexts_out[r] = a.contexts[r];
      }
    }
    __syncthreads();
  }
  if constexpr (UPDATE) {
    if (threadIdx.x == 0) {
      if (a.cu) a.cu[0] = 0;
      if (a.free_count_out) a.free_count_out[0] = count - used;
    }
  }
  if constexpr (FILL) {
    for (int t = blockIdx.x * MAPS_THREADS + threadIdx.x; t < a.T; t += gridDim.x * MAPS_THREADS) {
      int pos = 0, keep = -1;
      int64_t slot = -1;
      if (t < total) {
        int lo = 0, hi = a.N - 1; // the first request that ends behind t
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (ends[mid] > t) hi = mid;
          else lo = mid + 1;
        }
        const int begin = lo > 0 ? ends[lo - 1] : 0;
        pos = t + shift[lo];
        const int b = pos / B, held = blocks(begin + shift[lo]);
        int32_t* at = a.table + (int64_t)lo * a.max_blocks + b;
        int id;
        if (b < held) id = *at;
        else {
          id = a.free_list[count - 1 - (taken[lo] + b - held)];
          if (pos % B == 0) *at = id; // the token that enters a block
        }
        slot = (int64_t)id * B + pos % B;
        if ((pos + 1) % B == 0 && t + 1 < ends[lo]) keep = id;
      }
      if (a.positions) a.positions[t] = pos;
      if (a.token_slots) a.token_slots[t] = slot;
      if (a.slot_tok) a.slot_tok[t] = keep;
    }
  }
}

int launch_maps(const MapsArgs& a, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  constexpr int ALONE = 4 * MAPS_THREADS; // tokens that one workgroup fills with the rest
  if (a.T <= ALONE) {
    hipLaunchKernelGGL((k_maps<true, true>), dim3(1), dim3(MAPS_THREADS), 0, s, a);
    return (int)hipGetLastError();
  }
  const int groups = (a.T + MAPS_THREADS - 1) / MAPS_THREADS;
  hipLaunchKernelGGL((k_maps<true, false>), dim3((unsigned)(groups < 256 ? groups : 256)), dim3(MAPS_THREADS), 0, s, a);
  if (const int e = (int)hipGetLastError()) return e;
  hipLaunchKernelGGL((k_maps<false, true>), dim3(1), dim3(MAPS_THREADS), 0, s, a);
  return (int)hipGetLastError();
}

} // namespace gdn
