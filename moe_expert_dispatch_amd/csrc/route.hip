// Router: softmax over the expert logits and top-K selection, one wave per
// token.
//
// Source: vLLM ep_fused_moe_patch.py, module docstring "EP expert dispatch"
// (top-k routing yields the same global expert ids on every rank) and the
// FusedMoE constructor (top_k, renormalize). Selection compares the f32
// logits exactly; ties go to the lower expert id; -0.0 equals +0.0.
//
// Each lane holds E/64 (rounded up) logits in registers. Candidates carry a
// 64-bit key: the logit mapped to an order-preserving unsigned integer in the
// high word and (0xffffffff - id) in the low word, so one unsigned max picks
// the largest logit and, among equal logits, the lowest id. K rounds of a
// wave-wide max select the experts; the winner's owner lane clears its key.
//
// Up to 256 experts (K <= 8 or the lane count, no groups) a token gets
// L = 8, 16 or 32 lanes of a wave (at most 8 logits per lane) instead of a
// whole wave: lane q holds experts q, q + L, ..., sorted once in the lane,
// and each round's maximum is the DPP maximum of the lanes' first keys inside
// the group; the lane that held it moves its list up (route_lanes_kernel). Both forms give the same ids; the weights are
// the same softmax with the sums taken in a different order, and moe_route,
// moe_forward and the fused route + slot map of moe_forward all take the
// same form for a given shape, so their bits agree.
//
// Group-limited routing (the constructor's use_grouped_topk,
// num_expert_group and topk_group, which the pages only name; reading: the
// E experts form G consecutive groups scored by their largest logit): lane g
// gets group g's key (best ordered logit, 0xffffffff - g), topk_group rounds
// of a wave max pick the groups, and the keys of experts outside them are
// cleared before the K rounds. The softmax still runs over all E experts.
#include "route_token.h"

namespace moe {
namespace {

template <int L, int EPL, bool MAP>
__global__ __launch_bounds__(256) void route_lanes_kernel(const float* __restrict__ logits,
                                                          int T, int E, int K, int renorm,
                                                          int32_t* __restrict__ ids,
                                                          float* __restrict__ w, MapOut mo) {
  const int q = threadIdx.x & (L - 1);
  const uint32_t t = folded_block() * (256 / L) + threadIdx.x / L;
  const bool live = t < (uint32_t)T;
  int id;
  float p;
  route_token<L, EPL>(logits + (size_t)(live ? t : 0) * E, live, E, K, renorm, q, &id, &p);
  if (live && q < K) {
    const int pi = t * K + q;
    ids[pi] = id;
    w[pi] = p;
    if constexpr (MAP)
      map_pair(pi, t, id, p, mo.start, mo.E_local, mo.rep_off, mo.rep_slots, mo.S, mo.slot,
               mo.w_masked, mo.mask);
  }
}

// A plan in one block, for the few pairs of a decoding batch (P <=
// kPlanPairs): the counting sort of launch_permute with the same results, and
// before it, where the block's lanes hold all tokens at once (L > 1), routing
// and slot map. L == 1: the slot map is given. A wave holds 64 pairs in pair
// order; a pair's rank in its slot is the number of lower lanes with the same
// slot (one ballot per bit of the slot id) plus what the earlier waves hold
// of it (counts in LDS).
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kWave;
static_assert(kPlanThreads >= MOE_MAX_SLOTS && kPlanThreads >= kPlanPairs,
              "a thread for every slot and pair");

template <int L, int EPL>
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(
    const float* __restrict__ logits, int T, int E, int K, int renorm, MapOut mo,
    int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_pairs,
    int32_t* __restrict__ pair_row) {
  extern __shared__ int32_t wave_count[];  // [waves with pairs][S]
  __shared__ int32_t pair_slot[kPlanPairs];  // -1: not included
  __shared__ int32_t first[MOE_MAX_SLOTS];
  __shared__ int32_t wsum[kPlanWaves];
  const int tid = threadIdx.x;
  const int lane = lane_id();
  const int wave = tid / kWave;
  const int P = T * K;
  const int S = mo.S;
  const int nw = ceil_div(P, kWave);
  for (int i = tid; i < nw * S; i += kPlanThreads) wave_count[i] = 0;
  if constexpr (L > 1) {
    const int q = tid & (L - 1);
    const int t = tid / L;
    const bool live = t < T;
    int id;
    float p;
    route_token<L, EPL>(logits + (size_t)(live ? t : 0) * E, live, E, K, renorm, q, &id, &p);
    if (live && q < K) {
      const int pi = t * K + q;
      const int s = map_pair(pi, t, id, p, mo.start, mo.E_local, mo.rep_off, mo.rep_slots, S,
                             mo.slot, mo.w_masked, mo.mask);
      pair_slot[pi] = id >= mo.start && id < mo.start + mo.E_local ? s : -1;
    }
  } else if (tid < P) {
    const int s = mo.slot[tid];
    pair_slot[tid] = mo.mask[tid] != 0 && s >= 0 && s < S ? s : -1;
  }
  __syncthreads();
  const int s = tid < P ? pair_slot[tid] : -1;
  const int sbits = S > 1 ? 32 - __clz(S - 1) : 0;
  uint64_t same = __ballot(s >= 0);
  for (int bit = 0; bit < sbits; ++bit) {
    const bool on = (s >> bit) & 1;
    const uint64_t ones = __ballot(s >= 0 && on);
    same &= on ? ones : ~ones;
  }
  const uint64_t below = same & lanemask_lt();
  if (s >= 0 && below == 0) wave_count[wave * S + s] = __popcll(same);
  __syncthreads();
  // exclusive scan of the slots' counts, a slot a thread
  int n = 0;
  if (tid < S)
    for (int v = 0; v < nw; ++v) n += wave_count[v * S + tid];
  int incl = n;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int v = __shfl_up(incl, o, kWave);
    if (lane >= o) incl += v;
  }
  if (lane == kWave - 1) wsum[wave] = incl;
  __syncthreads();
  int at = incl - n;
  for (int v = 0; v < wave; ++v) at += wsum[v];
  if (tid < S) {
    first[tid] = at;
    offsets[tid] = at;
    if (tid == S - 1) offsets[S] = at + n;
  }
  __syncthreads();
  if (tid < P) {
    int row = -1;
    if (s >= 0) {
      row = first[s] + __popcll(below);
      for (int v = 0; v < wave; ++v) row += wave_count[v * S + s];
      sorted_pairs[row] = tid;
    }
    pair_row[tid] = row;
  }
}

// G == 0: plain top-K over all experts; otherwise 1 <= TG <= G <= 64, E % G == 0.
// MAP: the slot map of each selected pair as well (as in the lane-group form).
template <int EPL, bool MAP>
__global__ __launch_bounds__(256) void route_kernel(const float* __restrict__ logits, int T,
                                                    int E, int K, int renorm, int G, int TG,
                                                    int32_t* __restrict__ ids,
                                                    float* __restrict__ w, MapOut mo) {
  const uint32_t t = folded_block() * (256 / kWave) + threadIdx.x / kWave;
  if (t >= (uint32_t)T) return;  // wave-uniform
  const int lane = lane_id();
  const float* row = logits + (size_t)t * E;

  float v[EPL];
  uint64_t key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + kWave * j;
    if (e < E) {
      v[j] = row[e];
      key[j] = ((uint64_t)ordered_bits(v[j]) << 32) | (0xffffffffu - (uint32_t)e);
    } else {
      v[j] = -INFINITY;
      key[j] = 0;  // never selected: every real candidate has a non-zero key
    }
  }

  if (G > 0) {
    const int Eg = E / G;
    int grp[EPL];  // group of each of the lane's experts (-1: none)
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + kWave * j;
      grp[j] = e < E ? e / Eg : -1;
    }
    uint64_t gkey = 0;
    for (int g = 0; g < G; ++g) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        if (grp[j] == g) {
          const uint32_t o = (uint32_t)(key[j] >> 32);
          m = o > m ? o : m;
        }
      }
      m = wave_max_u32(m);
      if (lane == g) gkey = ((uint64_t)m << 32) | (0xffffffffu - (uint32_t)g);
    }
    uint64_t keep = 0;  // selected groups, the same in every lane
    for (int r = 0; r < TG; ++r) {
      const uint64_t best = wave_max_u64(gkey);
      const int g = (int)(0xffffffffu - (uint32_t)best);
      keep |= 1ull << g;
      if (lane == g) gkey = 0;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (grp[j] >= 0 && !((keep >> grp[j]) & 1ull)) key[j] = 0;
  }

  // K rounds of wave max; lane k keeps the k-th selection.
  int my_id = 0;
  float my_logit = 0.f;
  for (int k = 0; k < K; ++k) {
    uint64_t best = key[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) best = key[j] > best ? key[j] : best;
    best = wave_max_u64(best);
    const int e = (int)(0xffffffffu - (uint32_t)best);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane + kWave * j == e) key[j] = 0;
    if (lane == k) {
      my_id = e;
      my_logit = from_ordered((uint32_t)(best >> 32));
    }
  }

  // Softmax with the top logit as the shift: m = max_e l_e.
  const float m = __shfl(my_logit, 0, kWave);
  float part = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    if (lane + kWave * j < E) part += expf(v[j] - m);
  const float denom = wave_sum(part);
  float p = (lane < K) ? expf(my_logit - m) / denom : 0.f;
  if (renorm) {
    const float s = wave_sum(p);
    p = p / s;
  }
  if (lane < K) {
    const int pi = t * K + lane;
    ids[pi] = my_id;
    w[pi] = p;
    if constexpr (MAP)
      map_pair(pi, t, my_id, p, mo.start, mo.E_local, mo.rep_off, mo.rep_slots, mo.S, mo.slot,
               mo.w_masked, mo.mask);
  }
}

template <int L, bool MAP>
void launch_lanes(const float* logits, int T, int E, int K, int renorm, int32_t* ids, float* w,
                  const MapOut& mo, hipStream_t stream) {
  const int epl = ceil_div(E, L);
  const dim3 grid = folded((T - 1) / (256 / L) + 1, 256);
  if (epl <= 1)
    route_lanes_kernel<L, 1, MAP><<<grid, 256, 0, stream>>>(logits, T, E, K, renorm, ids, w, mo);
  else if (epl <= 2)
    route_lanes_kernel<L, 2, MAP><<<grid, 256, 0, stream>>>(logits, T, E, K, renorm, ids, w, mo);
  else if (epl <= 4)
    route_lanes_kernel<L, 4, MAP><<<grid, 256, 0, stream>>>(logits, T, E, K, renorm, ids, w, mo);
  else
    route_lanes_kernel<L, 8, MAP><<<grid, 256, 0, stream>>>(logits, T, E, K, renorm, ids, w, mo);
}

// One wave per token (group-limited routing, more than 256 experts, K > 32).
template <bool MAP>
void launch_waves(const float* logits, int T, int E, int K, int renorm, int G, int TG,
                  int32_t* ids, float* w, const MapOut& mo, hipStream_t stream) {
  const dim3 block(256);
  const dim3 grid = folded((T - 1) / (256 / kWave) + 1, 256);
  const int epl = ceil_div(E, kWave);
  if (epl <= 1)
    route_kernel<1, MAP><<<grid, block, 0, stream>>>(logits, T, E, K, renorm, G, TG, ids, w, mo);
  else if (epl <= 2)
    route_kernel<2, MAP><<<grid, block, 0, stream>>>(logits, T, E, K, renorm, G, TG, ids, w, mo);
  else if (epl <= 4)
    route_kernel<4, MAP><<<grid, block, 0, stream>>>(logits, T, E, K, renorm, G, TG, ids, w, mo);
  else if (epl <= 8)
    route_kernel<8, MAP><<<grid, block, 0, stream>>>(logits, T, E, K, renorm, G, TG, ids, w, mo);
  else
    route_kernel<16, MAP><<<grid, block, 0, stream>>>(logits, T, E, K, renorm, G, TG, ids, w,
                                                      mo);
}

template <bool MAP>
void launch_lanes_any(int L, const float* logits, int T, int E, int K, int renorm, int32_t* ids,
                      float* w, const MapOut& mo, hipStream_t stream) {
  if (L == 8)
    launch_lanes<8, MAP>(logits, T, E, K, renorm, ids, w, mo, stream);
  else if (L == 16)
    launch_lanes<16, MAP>(logits, T, E, K, renorm, ids, w, mo, stream);
  else
    launch_lanes<32, MAP>(logits, T, E, K, renorm, ids, w, mo, stream);
}

size_t plan_lds(int P, int S) { return (size_t)ceil_div(P, kWave) * S * sizeof(int32_t); }

template <int L>
void launch_plan_lanes(const float* logits, int T, int E, int K, int renorm, const MapOut& mo,
                       int32_t* offsets, int32_t* sorted_pairs, int32_t* pair_row,
                       hipStream_t stream) {
  auto go = [&](auto epl) {
    plan_kernel<L, decltype(epl)::value><<<1, kPlanThreads, plan_lds(T * K, mo.S), stream>>>(
        logits, T, E, K, renorm, mo, offsets, sorted_pairs, pair_row);
  };
  const int epl = ceil_div(E, L);
  if (epl <= 1)
    go(std::integral_constant<int, 1>{});
  else if (epl <= 2)
    go(std::integral_constant<int, 2>{});
  else if (epl <= 4)
    go(std::integral_constant<int, 4>{});
  else
    go(std::integral_constant<int, 8>{});
}

}  // namespace

// Lanes per token for the grouped-lane router (at most 8 logits per lane and
// K <= L), or 0 where the wave-per-token kernel runs (group-limited routing,
// more than 256 experts, K > 32).
int route_lanes(int E, int K, int G) {
  if (G != 0 || E > 256 || K > 32) return 0;
  if (E <= 64 && K <= 8) return 8;
  if (E <= 128 && K <= 16) return 16;
  return 32;
}

moe_status_t launch_route_map(const float* logits, int T, int E, int K, int renorm, int G,
                              int TG, int32_t* ids, float* w, int start, int E_local,
                              const int32_t* rep_off, const int32_t* rep_slots, int S,
                              int32_t* slot, float* w_masked, uint8_t* mask,
                              hipStream_t stream) {
  if (T == 0) return MOE_OK;
  const int L = route_lanes(E, K, G);
  const MapOut mo{start, E_local, S, rep_off, rep_slots, slot, w_masked, mask};
  if (L == 0)
    launch_waves<true>(logits, T, E, K, renorm, G, TG, ids, w, mo, stream);
  else
    launch_lanes_any<true>(L, logits, T, E, K, renorm, ids, w, mo, stream);
  return launch_status();
}

moe_status_t launch_route(const float* logits, int T, int E, int K, int renorm, int G, int TG,
                          int32_t* ids, float* w, hipStream_t stream) {
  if (T == 0) return MOE_OK;
  if (const int L = route_lanes(E, K, G)) {
    launch_lanes_any<false>(L, logits, T, E, K, renorm, ids, w, MapOut{}, stream);
    return launch_status();
  }
  launch_waves<false>(logits, T, E, K, renorm, G, TG, ids, w, MapOut{}, stream);
  return launch_status();
}

moe_status_t launch_plan(const float* logits, int T, int E, int K, int renorm, int G, int TG,
                         int32_t* ids, float* w, int start, int E_local, const int32_t* rep_off,
                         const int32_t* rep_slots, int S, int32_t* slot, float* w_masked,
                         uint8_t* mask, int32_t* offsets, int32_t* sorted_pairs,
                         int32_t* pair_row, hipStream_t stream) {
  const MapOut mo{start, E_local, S, rep_off, rep_slots, slot, w_masked, mask};
  const int L = logits != nullptr ? route_lanes(E, K, G) : 0;
  if (L > 0 && T * L <= kPlanThreads) {
    if (L == 8)
      launch_plan_lanes<8>(logits, T, E, K, renorm, mo, offsets, sorted_pairs, pair_row, stream);
    else if (L == 16)
      launch_plan_lanes<16>(logits, T, E, K, renorm, mo, offsets, sorted_pairs, pair_row, stream);
    else
      launch_plan_lanes<32>(logits, T, E, K, renorm, mo, offsets, sorted_pairs, pair_row, stream);
    return launch_status();
  }
  const moe_status_t st =
      logits != nullptr
          ? launch_route_map(logits, T, E, K, renorm, G, TG, ids, w, start, E_local, rep_off,
                             rep_slots, S, slot, w_masked, mask, stream)
          : launch_slot_map(ids, w, T, K, start, E_local, rep_off, rep_slots, S, slot, w_masked,
                            mask, stream);
  if (st != MOE_OK) return st;
  plan_kernel<1, 1><<<1, kPlanThreads, plan_lds(T * K, S), stream>>>(
      nullptr, T, E, K, renorm, mo, offsets, sorted_pairs, pair_row);
  return launch_status();
}

}  // namespace moe
