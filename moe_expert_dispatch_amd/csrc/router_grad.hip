// The router's balance loss, per-expert counts, and the gradient of routing
// weights and loss with respect to the logits.
//
//   p_t = softmax(logits_t) over the valid tokens t, n of them
//   counts_e = number of valid pairs with ids = e,  f_e = counts_e / (n K)
//   P_e = (1/n) sum_t p_te,  loss = coef E sum_e f_e P_e
//   d loss / d logits_te = coef (E / n) p_te (f_e - sum_j f_j p_tj)
//     (the counts are piecewise constant in the logits: no gradient)
//   routing weights w_k = p_{ids_k}:
//     d_te = p_te (sum_{k: ids_k = e} dw_k - sum_k p_{ids_k} dw_k)
//   renormalised, w = softmax over the K selected logits:
//     d_te = sum_{k: ids_k = e} w_k (dw_k - sum_j w_j dw_j)
//
// L lanes of a wave hold one token (expert e in lane e mod L), as in the
// router. The loss walks tokens with a fixed grid and sums in f32 in a fixed
// order: per lane over its tokens, per block over its lane groups, then in
// f64 over the blocks, so the result does not depend on scheduling. Counts
// are integers (LDS atomics). The backward pass reads each logit once and
// writes each gradient once; softmax, both dot products and the scatter of
// the K weights stay in registers.
#include <algorithm>

#include "common.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 256;

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L == kWave)
    return wave_sum(v);
  else
    return group_sum<L>(v);
}

template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __uint_as_float(dpp_u32<decltype(ctrl)::value>(__float_as_uint(x)));
  };
  v = fmaxf(v, dpp(v, std::integral_constant<int, kDppQuad1032>{}));
  v = fmaxf(v, dpp(v, std::integral_constant<int, kDppQuad2301>{}));
  v = fmaxf(v, dpp(v, std::integral_constant<int, kDppRowHalfMirror>{}));
  if constexpr (L >= 16) v = fmaxf(v, dpp(v, std::integral_constant<int, kDppRowMirror>{}));
  if constexpr (L >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v),
                                                    false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  }
  if constexpr (L == kWave) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v),
                                                    false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  }
  return v;
}

// Softmax of one token's logits, in place; returns nothing where the row has
// no finite logit (every p is 0 then). Every lane of the wave takes part.
template <int L, int EPL>
__device__ __forceinline__ void token_softmax(const float* __restrict__ row, int E, int q,
                                              bool live, float (&p)[EPL], float* shift,
                                              float* denom) {
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = q + L * j;
    p[j] = live && e < E ? row[e] : -INFINITY;
  }
  float m = p[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) m = fmaxf(m, p[j]);
  m = lanes_max<L>(m);
  const float s = m == -INFINITY ? 0.f : m;  // -inf - 0 instead of -inf - -inf
  float part = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    p[j] = expf(p[j] - s);
    part += p[j];
  }
  const float d = lanes_sum<L>(part);
  const float inv = d > 0.f ? 1.0f / d : (d == 0.f ? 0.f : d);
#pragma unroll
  for (int j = 0; j < EPL; ++j) p[j] *= inv;
  *shift = s;
  *denom = d;
}

template <int L, int EPL>
__global__ __launch_bounds__(kThreads) void balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ token_mask, int T, int E, int K, float* __restrict__ part_p,
    int32_t* __restrict__ part_c) {
  constexpr int kGroups = kThreads / L;
  __shared__ int32_t cnt[L * EPL + 1];
  __shared__ float sums[kGroups][L * EPL];
  for (int i = threadIdx.x; i < L * EPL + 1; i += kThreads) cnt[i] = 0;
  __syncthreads();
  const int q = threadIdx.x & (L - 1);
  const int grp = threadIdx.x / L;
  float acc[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
  int valid = 0;
  // every lane of a wave runs the same number of rounds: the reductions read
  // all lanes
  for (int t0 = blockIdx.x * kGroups; t0 < T; t0 += gridDim.x * kGroups) {
    const int t = t0 + grp;
    const bool live = t < T && (token_mask == nullptr || token_mask[t] != 0);
    float p[EPL], shift, denom;
    token_softmax<L, EPL>(logits + (size_t)(live ? t : 0) * E, E, q, live, p, &shift, &denom);
    if (live) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) acc[j] += p[j];
      ++valid;
      if (q < K) {
        const int id = ids[(size_t)t * K + q];
        if (id >= 0 && id < E) atomicAdd(&cnt[id], 1);
      }
    }
  }
  if (q == 0 && valid > 0) atomicAdd(&cnt[L * EPL], valid);
#pragma unroll
  for (int j = 0; j < EPL; ++j) sums[grp][q + L * j] = acc[j];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float s = 0.f;
    for (int g = 0; g < kGroups; ++g) s += sums[g][e];
    part_p[(size_t)blockIdx.x * E + e] = s;
    part_c[(size_t)blockIdx.x * (E + 1) + e] = cnt[e];
  }
  if (threadIdx.x == 0) part_c[(size_t)blockIdx.x * (E + 1) + E] = cnt[L * EPL];
}

constexpr int kFinalThreads = 1024;

// One block: the blocks' partial sums in order, the means, and the loss.
__global__ __launch_bounds__(kFinalThreads) void balance_final_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c, int nblk, int E, int K,
    int ways, float coef, int32_t* __restrict__ counts, float* __restrict__ prob,
    float* __restrict__ loss) {
  __shared__ double sp[kFinalThreads];
  __shared__ int32_t sc[kFinalThreads];
  __shared__ int32_t n_all;
  const int tid = threadIdx.x;
  // ways threads per expert, each over every ways-th block
  const int Ep = kFinalThreads / ways;
  const int e = tid % Ep, way = tid / Ep;
  int32_t nv = 0;
  for (int b = tid; b < nblk; b += kFinalThreads) nv += part_c[(size_t)b * (E + 1) + E];
  sc[tid] = nv;
  __syncthreads();
  for (int o = kFinalThreads / 2; o > 0; o >>= 1) {
    if (tid < o) sc[tid] += sc[tid + o];
    __syncthreads();
  }
  if (tid == 0) n_all = sc[0];
  __syncthreads();
  const int n = n_all;
  double s = 0.0;
  int32_t c = 0;
  if (e < E)
    for (int b = way; b < nblk; b += ways) {
      s += (double)part_p[(size_t)b * E + e];
      c += part_c[(size_t)b * (E + 1) + e];
    }
  sp[tid] = s;
  sc[tid] = c;
  __syncthreads();
  double term = 0.0;
  if (way == 0 && e < E) {
    for (int w = 1; w < ways; ++w) {
      s += sp[w * Ep + e];
      c += sc[w * Ep + e];
    }
    const double mean = n > 0 ? s / n : 0.0;
    counts[e] = c;
    prob[e] = (float)mean;
    term = n > 0 ? mean * ((double)c / ((double)n * K)) : 0.0;
  }
  __syncthreads();
  sp[tid] = term;
  __syncthreads();
  for (int o = kFinalThreads / 2; o > 0; o >>= 1) {
    if (tid < o) sp[tid] += sp[tid + o];
    __syncthreads();
  }
  if (tid == 0) {
    counts[E] = n;
    *loss = (float)((double)coef * E * sp[0]);
  }
}

template <int L, int EPL>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, const uint8_t* __restrict__ token_mask,
    const int32_t* __restrict__ counts, const float* __restrict__ dloss, int T, int E, int K,
    int renorm, float coef, float* __restrict__ dlogits) {
  constexpr int kGroups = kThreads / L;
  const int q = threadIdx.x & (L - 1);
  const int t = blockIdx.x * kGroups + threadIdx.x / L;
  const bool inside = t < T;
  const bool live = inside && (token_mask == nullptr || token_mask[t] != 0);
  const float* row = logits + (size_t)(live ? t : 0) * E;
  float p[EPL], shift, denom;
  token_softmax<L, EPL>(row, E, q, live, p, &shift, &denom);
  float d[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) d[j] = 0.f;

  if (dw != nullptr) {
    int id = -1;
    float z = -INFINITY, up = 0.f;
    if (live && q < K) {
      const int v = ids[(size_t)t * K + q];
      if (v >= 0 && v < E) {
        id = v;
        z = row[v];
        up = dw[(size_t)t * K + q];
      }
    }
    float s = shift;
    if (renorm) {  // the selected logits' own shift: their weights never all underflow
      s = lanes_max<L>(z);
      s = s == -INFINITY ? 0.f : s;
    }
    float w = expf(z - s);
    const float total = renorm ? lanes_sum<L>(w) : denom;
    w = total > 0.f ? w / total : (total == 0.f ? 0.f : total);
    const float dot = lanes_sum<L>(w * up);
    const float mine = renorm ? w * (up - dot) : w * up;
    if (!renorm) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) d[j] = -p[j] * dot;
    }
    for (int k = 0; k < K; ++k) {
      const int e = __shfl(id, k, L);
      const float g = __shfl(mine, k, L);
#pragma unroll
      for (int j = 0; j < EPL; ++j) d[j] += e == q + L * j ? g : 0.f;
    }
  }
  if (counts != nullptr) {
    const int n = counts[E];
    const float share = n > 0 ? 1.0f / ((float)n * (float)K) : 0.f;
    float f[EPL], part = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = q + L * j;
      f[j] = e < E ? (float)counts[e] * share : 0.f;
      part = fmaf(f[j], p[j], part);
    }
    const float mean = lanes_sum<L>(part);
    const float c = (dloss != nullptr ? *dloss : 1.0f) * coef * (float)E * share * (float)K;
#pragma unroll
    for (int j = 0; j < EPL; ++j) d[j] = fmaf(c * p[j], f[j] - mean, d[j]);
  }
  if (inside) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = q + L * j;
      if (e < E) dlogits[(size_t)t * E + e] = live ? d[j] : 0.f;
    }
  }
}

// Lanes per token: at most 8 logits a lane up to 512 experts, 16 above, and a
// lane for each of the K selected experts.
int lanes_for(int E, int K) {
  if (E <= 64 && K <= 8) return 8;
  if (E <= 128 && K <= 16) return 16;
  if (E <= 256) return 32;
  return kWave;
}

template <typename F>
void with_lanes(int E, int K, F&& f) {
  using std::integral_constant;
  const int L = lanes_for(E, K);
  const int epl = ceil_div(E, L);
  auto pick = [&](auto l) {
    if (epl <= 1)
      f(l, integral_constant<int, 1>{});
    else if (epl <= 2)
      f(l, integral_constant<int, 2>{});
    else if (epl <= 4)
      f(l, integral_constant<int, 4>{});
    else
      f(l, integral_constant<int, 8>{});
  };
  if (L == 8)
    pick(integral_constant<int, 8>{});
  else if (L == 16)
    pick(integral_constant<int, 16>{});
  else if (L == 32)
    pick(integral_constant<int, 32>{});
  else if (epl <= 8)
    f(integral_constant<int, kWave>{}, integral_constant<int, 8>{});
  else
    f(integral_constant<int, kWave>{}, integral_constant<int, 16>{});
}

int balance_blocks(int T, int E, int K) {
  return std::max(1, std::min(kMaxBlocks, ceil_div(T, kThreads / lanes_for(E, K))));
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int K) {
  return (size_t)balance_blocks(T, E, K) * (size_t)(2 * E + 1) * 4;
}

moe_status_t launch_balance_loss(const float* logits, const int32_t* ids,
                                 const uint8_t* token_mask, int T, int E, int K, float coef,
                                 int32_t* counts, float* prob, float* loss, void* ws,
                                 hipStream_t stream) {
  const int nblk = balance_blocks(T, E, K);
  float* part_p = static_cast<float*>(ws);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + (size_t)nblk * E);
  with_lanes(E, K, [&](auto l, auto epl) {
    balance_partial_kernel<decltype(l)::value, decltype(epl)::value>
        <<<nblk, kThreads, 0, stream>>>(logits, ids, token_mask, T, E, K, part_p, part_c);
  });
  int ways = 1;
  while (2 * ways * E <= kFinalThreads && ways < 256) ways *= 2;
  balance_final_kernel<<<1, kFinalThreads, 0, stream>>>(part_p, part_c, nblk, E, K, ways, coef,
                                                        counts, prob, loss);
  return launch_status();
}

moe_status_t launch_route_backward(const float* logits, const int32_t* ids, const float* dw,
                                   const uint8_t* token_mask, const int32_t* counts,
                                   const float* dloss, int T, int E, int K, int renorm,
                                   float coef, float* dlogits, hipStream_t stream) {
  if (T == 0) return MOE_OK;
  with_lanes(E, K, [&](auto l, auto epl) {
    constexpr int L = decltype(l)::value;
    route_backward_kernel<L, decltype(epl)::value>
        <<<ceil_div(T, kThreads / L), kThreads, 0, stream>>>(
            logits, ids, dw, token_mask, counts, dloss, T, E, K, renorm, coef, dlogits);
  });
  return launch_status();
}

}  // namespace moe
