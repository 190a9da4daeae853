// The selection and the weights of one token by a group of lanes: used by the
// router's kernels (route.hip, where the method is described) and by the
// products that route their own pairs (mxfp4.hip).
#pragma once
#include "common.h"

namespace moe {

__device__ __forceinline__ uint32_t ordered_bits(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;  // NaN ranks below everything
  if ((u & 0x7fffffffu) == 0u) u = 0u;              // -0.0 -> +0.0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Inverse of ordered_bits for non-NaN keys (-0.0 comes back as +0.0, which
// gives the same exponentials).
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// Sorts n <= 8 keys into descending order with a comparator network
// (Batcher's odd-even merge sort: 1, 5 or 19 compare-exchanges).
template <int N>
__device__ __forceinline__ void sort_desc(uint64_t (&k)[N]) {
  auto cx = [&](int a, int b) {
    const uint64_t hi = k[a] > k[b] ? k[a] : k[b];
    const uint64_t lo = k[a] > k[b] ? k[b] : k[a];
    k[a] = hi;
    k[b] = lo;
  };
  if constexpr (N == 2) {
    cx(0, 1);
  } else if constexpr (N == 4) {
    cx(0, 1); cx(2, 3); cx(0, 2); cx(1, 3); cx(1, 2);
  } else if constexpr (N == 8) {
    cx(0, 1); cx(2, 3); cx(4, 5); cx(6, 7);
    cx(0, 2); cx(1, 3); cx(4, 6); cx(5, 7);
    cx(1, 2); cx(5, 6);
    cx(0, 4); cx(1, 5); cx(2, 6); cx(3, 7);
    cx(2, 4); cx(3, 5);
    cx(1, 2); cx(3, 4); cx(5, 6);
  } else {
    static_assert(N == 1, "1, 2, 4 or 8 keys per lane");
  }
}

// The selection of one token by the L lanes of its group (q: the lane in it):
// lane q < K ends with the q-th expert and its weight. EPL logits per lane (a
// power of two); K <= L, E <= L * EPL. Lanes of tokens that do not exist (not
// live) carry empty keys, but stay active, so every DPP step reads live lanes.
template <int L, int EPL>
__device__ __forceinline__ void route_token(const float* __restrict__ row, bool live, int E, int K,
                                            int renorm, int q, int* id, float* weight) {
  float v[EPL];
  uint64_t key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = q + L * j;
    if (live && e < E) {
      v[j] = row[e];
      key[j] = ((uint64_t)ordered_bits(v[j]) << 32) | (0xffffffffu - (uint32_t)e);
    } else {
      v[j] = -INFINITY;
      key[j] = 0;
    }
  }

  // K rounds; lane k of the group keeps the k-th selection's key. The
  // lane's keys are sorted once, so a round's candidate is key[0] and only
  // the lane holding the group's maximum (keys are unique) moves its list up.
  sort_desc<EPL>(key);
  uint64_t my_key = 0;
  uint64_t top = 0;
  for (int k = 0; k < K; ++k) {
    const uint64_t best = group_max_u64<L>(key[0]);
    // all ones in the lane that held it (as a bit mask: one select per word)
    const uint64_t mv = 0ull - (uint64_t)(key[0] == best);
#pragma unroll
    for (int j = 0; j + 1 < EPL; ++j) key[j] = (key[j + 1] & mv) | (key[j] & ~mv);
    key[EPL - 1] &= ~mv;
    if (q == k) my_key = best;
    if (k == 0) top = best;
  }

  // Softmax with the top logit as the shift.
  const float m = from_ordered((uint32_t)(top >> 32));
  float part = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    if (q + L * j < E) part += expf(v[j] - m);
  const float denom = group_sum<L>(part);
  float p = (q < K) ? expf(from_ordered((uint32_t)(my_key >> 32)) - m) / denom : 0.f;
  if (renorm) {
    const float s = group_sum<L>(p);
    p = p / s;
  }
  *id = (int)(0xffffffffu - (uint32_t)my_key);
  *weight = p;
}

// The slot of pair p (token p / topk, its selection p % topk), routed by a
// wave with the L lanes of its groups all working on that token; -1 where the
// pair is another rank's or has no slot. write: the slot map's entry as well.
// EPL = 8 for every E: lists filled up with empty keys, and sums that skip
// them, give the bits of the shorter ones.
template <int L>
__device__ __forceinline__ int route_pair(const PairRouting& in, int p, int topk, bool write) {
  const int t = p / topk;
  const int q = lane_id() & (L - 1);
  int id;
  float w;
  route_token<L, 8>(in.logits + (size_t)t * in.E, true, in.E, topk, in.renorm, q, &id, &w);
  const int k = p - t * topk;
  const MapOut& mo = in.map;
  int s = -1;
  if (lane_id() == k) {
    if (write)
      s = map_pair(p, t, id, w, mo.start, mo.E_local, mo.rep_off, mo.rep_slots, mo.S, mo.slot,
                   mo.w_masked, mo.mask);
    else
      s = map_slot(t, id, mo.start, mo.E_local, mo.rep_off, mo.rep_slots, mo.S);
    if (id < mo.start || id >= mo.start + mo.E_local) s = -1;
  }
  return __builtin_amdgcn_readlane(s, __builtin_amdgcn_readfirstlane(k));
}

}  // namespace moe
