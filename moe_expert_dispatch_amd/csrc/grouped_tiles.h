// What the grouped products of the gradient share: row tiles of all slots,
// numbered in a prefix that every block builds for itself, and the order in
// which blocks take work items.
#pragma once

#include "common.h"
#include "item_order.h"
#include "split_rows.h"

namespace moe {

// Block-uniform values read from LDS or memory, moved to scalar registers.
__device__ __forceinline__ int uniform_i32(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A slot's rows [lo, hi) from its entries of offsets, kept inside the buffers
// whatever the device data says.
__device__ __forceinline__ void slot_rows(const int32_t* __restrict__ offsets, int s, int max_rows,
                                          int* lo, int* hi) {
  const int a = offsets[s], b = offsets[s + 1];
  *lo = a < 0 ? 0 : min(a, max_rows);
  *hi = b < *lo ? *lo : min(b, max_rows);
}

// tp[0..S] = prefix over slots of ceil(rows / BM), in LDS. Every one of the
// block's NT threads calls it (it contains barriers); scratch holds NT ints.
template <int NT, int BM>
__device__ void tile_prefix(const int32_t* __restrict__ offsets, int S, int max_rows, int32_t* tp,
                            int32_t* scratch) {
  const int tid = threadIdx.x;
  const int per = ceil_div(S, NT);
  const int first = min(tid * per, S), last = min(first + per, S);
  auto tiles = [&](int s) {
    int lo, hi;
    slot_rows(offsets, s, max_rows, &lo, &hi);
    return (hi - lo) / BM + ((hi - lo) % BM != 0);
  };
  int sum = 0;
  for (int s = first; s < last; ++s) sum += tiles(s);
  scratch[tid] = sum;
  __syncthreads();
  for (int off = 1; off < NT; off <<= 1) {
    const int v = tid >= off ? scratch[tid - off] : 0;
    __syncthreads();
    scratch[tid] += v;
    __syncthreads();
  }
  int run = scratch[tid] - sum;
  for (int s = first; s < last; ++s) {
    tp[s] = run;
    run += tiles(s);
  }
  if (tid == NT - 1) tp[S] = scratch[NT - 1];
  __syncthreads();
}

// The slot of row tile rt: the largest s with tp[s] <= rt (it has rows).
__device__ __forceinline__ int tile_slot(const int32_t* tp, int S, int rt) {
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tp[mid] <= rt) lo = mid; else hi = mid;
  }
  return lo;
}

// With one block a compute unit, blocks b, b + 8, .. run on one XCD: it takes
// neighbouring items, which share operands in its L2.
__device__ __forceinline__ int first_item(int b, int G) {
  return G % 8 == 0 ? (b % 8) * (G / 8) + b / 8 : b;
}

}  // namespace moe
