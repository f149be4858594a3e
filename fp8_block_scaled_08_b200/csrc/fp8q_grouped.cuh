// Ragged groups of token rows (the experts of a layer with one weight per expert), shared
// by the grouped GEMMs and quantizers.
//
// offsets[0 .. E] (int32, in device memory) gives expert e the rows offsets[e] ..
// offsets[e + 1] - 1. The kernels read it themselves, so that no call waits for the host
// to learn the routing; every CTA builds the same table of E + 1 running counts in shared
// memory at its start and finds the expert of a tile by binary search. Nothing that a
// kernel reads or writes may depend on the offsets being sane: they are clamped to
// [0, limit] and to their running maximum, and the first CTA reports a clamped entry in
// the device error word.
#pragma once

#include "fp8q_device.cuh"
#include "fp8q_host.h"

namespace fp8q {

// off[0 .. E] = the clamped offsets; first[e] = the number of units (row blocks) of the
// experts before e, with count(lo, hi) units for rows [lo, hi). Called by every thread of
// the CTA; the caller synchronises the CTA before it reads the table. The loads are issued
// by all threads at once (a latency, not E of them); one warp then does the two scans.
template <class Count>
__device__ __forceinline__ void group_table_fill(int* off, int* first,
                                                 const int32_t* offsets, int E,
                                                 int limit, unsigned* err, Count count) {
  for (int i = threadIdx.x; i <= E; i += blockDim.x) off[i] = ld_after_wait(offsets + i);
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int lane = static_cast<int>(lane_id());
  bool bad = false;
  int carry = 0;
  for (int b = 0; b <= E; b += 32) {
    const int i = b + lane;
    const int raw = i <= E ? off[i] : 0;
    int v = min(max(raw, carry), limit);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v = max(v, u);
    }
    carry = __shfl_sync(0xFFFFFFFFu, v, 31);
    if (i <= E) {
      bad |= v != raw;
      off[i] = v;
    }
  }
  if (bad && blockIdx.x == 0) atomicOr(err, kErrOffsets);
  __syncwarp();
  int total = 0;
  for (int b = 0; b < E; b += 32) {
    const int i = b + lane;
    int v = i < E ? count(off[i], off[i + 1]) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v += u;
    }
    if (i < E) first[i + 1] = total + v;
    total += __shfl_sync(0xFFFFFFFFu, v, 31);
  }
  if (lane == 0) first[0] = 0;
}

// The expert of unit u (first[e] <= u < first[e + 1]), for 0 <= u < first[E].
__device__ __forceinline__ int group_find(const int* first, int E, int u) {
  int lo = 0, hi = E;  // first[lo] <= u < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Shared memory of the table.
constexpr uint32_t group_table_bytes(int E) { return 2u * (static_cast<uint32_t>(E) + 1u) * 4u; }

}  // namespace fp8q
