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
// L lanes of a wave hold one token, as in the router: lane q the experts
// 4 (q + L i) .. + 3 where rows are whole aligned 16-byte vectors, else
// q + L i. The loss walks tokens with a fixed grid, two at a time, and sums
// in f32 in a fixed order: per lane over its tokens, over the lane groups of
// a wave, over a block's waves, then in f64 over the blocks, so the result
// does not depend on scheduling. Counts are integers (LDS atomics). The
// backward pass reads each logit once and writes each gradient once; softmax
// and both dot products stay in registers, the K selected terms reach their
// lanes through LDS.
//
// Bound by the logits' and gradients' bytes. 65536 tokens x 256 experts,
// top-8: sums 19 us (3.5 TB/s; one token at a time on 4 waves a compute unit
// 46), their fold and the outputs 9, backward 31 us (4.5 TB/s; with a compare
// and select per selected expert and logit instead of the LDS row 38). At a
// few hundred tokens three launches' latency is all there is, so up to four
// rounds of tokens one block does the loss alone.
#include <algorithm>

#include "common.h"

namespace moe {
namespace {

constexpr int kLossThreads = 1024;
constexpr int kLossWaves = kLossThreads / kWave;
constexpr int kLossRounds = 4;   // rounds of tokens that one block takes before there are more
constexpr int kMaxBlocks = 256;
constexpr int kGradThreads = 256;
constexpr int kGradBlocks = 2048;

// Expert j of lane q's EPL, or at least E where it has none.
template <int L, int EPL, bool VEC>
__device__ __forceinline__ int expert_of(int q, int j) {
  return VEC ? 4 * (q + L * (j >> 2)) + (j & 3) : q + L * j;
}

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

// One token's logits: -inf where there is no expert or no token.
template <int L, int EPL, bool VEC>
__device__ __forceinline__ void load_token(const float* __restrict__ row, int E, int q, bool live,
                                           float (&p)[EPL]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < EPL; j += 4) {
      const int e = expert_of<L, EPL, VEC>(q, j);
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (live && e < E) v = *reinterpret_cast<const float4*>(row + e);
      p[j] = v.x;
      p[j + 1] = v.y;
      p[j + 2] = v.z;
      p[j + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = expert_of<L, EPL, VEC>(q, j);
      p[j] = live && e < E ? row[e] : -INFINITY;
    }
  }
}

// Softmax of one token's logits, in place; every p is 0 where the row has no
// finite logit. Every lane of the wave takes part.
template <int L, int EPL>
__device__ __forceinline__ void token_softmax(float (&p)[EPL], float* shift, float* denom) {
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

// Sum of a value of every thread over the block, in the threads' order
// halved; every thread has to call it. buf holds kLossThreads values.
__device__ __forceinline__ double block_sum(double v, double* buf) {
  const int tid = threadIdx.x;
  buf[tid] = v;
  __syncthreads();
  for (int o = kLossThreads / 2; o > 0; o >>= 1) {
    if (tid < o) buf[tid] += buf[tid + o];
    __syncthreads();
  }
  return buf[0];
}

// Expert e's outputs from its sums over all tokens, and the loss.
__device__ __forceinline__ void finish_loss(double s, int32_t c, int n, bool mine, int e, int E,
                                            int K, float coef, int32_t* counts, float* prob,
                                            float* loss, double* buf) {
  double term = 0.0;
  if (mine) {
    const double mean = n > 0 ? s / n : 0.0;
    counts[e] = c;
    prob[e] = (float)mean;
    term = n > 0 ? mean * ((double)c / ((double)n * K)) : 0.0;
  }
  const double sum = block_sum(term, buf);
  if (threadIdx.x == 0) {
    counts[E] = n;
    *loss = (float)((double)coef * E * sum);
  }
}

// ONE: the only block, which writes the outputs itself; else the block's sums
// and counts go to part[block][E + 1] (the last entry: the valid tokens).
template <int L, int EPL, bool VEC, bool ONE>
__global__ __launch_bounds__(kLossThreads) void balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ token_mask, int T, int E, int K, float2* __restrict__ part,
    float coef, int32_t* __restrict__ counts, float* __restrict__ prob,
    float* __restrict__ loss) {
  constexpr int kGroups = kLossThreads / L;
  constexpr int kWidth = L * EPL;
  __shared__ int32_t cnt[kWidth + 1];
  __shared__ float sums[kLossWaves][kWidth];
  for (int i = threadIdx.x; i < kWidth + 1; i += kLossThreads) cnt[i] = 0;
  __syncthreads();
  const int q = threadIdx.x & (L - 1);
  const int grp = threadIdx.x / L;
  float acc[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
  int valid = 0;
  // two tokens at a time; every lane of a wave runs the same number of rounds,
  // since the reductions read all lanes
  const uint32_t n = (uint32_t)T;  // unsigned: a step past the end does not overflow
  const uint32_t stride = gridDim.x * kGroups;
  for (uint32_t t0 = blockIdx.x * kGroups; t0 < n; t0 += 2 * stride) {
    const uint32_t t[2] = {t0 + grp, t0 + stride + grp};
    bool live[2];
    float p[2][EPL], shift, denom;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      live[u] = t[u] < n && (token_mask == nullptr || token_mask[t[u]] != 0);
      load_token<L, EPL, VEC>(logits + (size_t)(live[u] ? t[u] : 0) * E, E, q, live[u], p[u]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (live[u]) {
        ++valid;
        if (q < K) {
          const int id = ids[(size_t)t[u] * K + q];
          if (id >= 0 && id < E) atomicAdd(&cnt[id], 1);
        }
      }
      token_softmax<L, EPL>(p[u], &shift, &denom);
#pragma unroll
      for (int j = 0; j < EPL; ++j) acc[j] += live[u] ? p[u][j] : 0.f;
    }
  }
  if (q == 0 && valid > 0) atomicAdd(&cnt[kWidth], valid);
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
#pragma unroll
    for (int o = L; o < kWave; o <<= 1) acc[j] += __shfl_xor(acc[j], o, kWave);
    const int e = expert_of<L, EPL, VEC>(q, j);
    if (lane_id() < L) sums[threadIdx.x / kWave][e] = acc[j];
  }
  __syncthreads();
  if constexpr (ONE) {
    __shared__ double buf[kLossThreads];
    const int e = threadIdx.x;
    double s = 0.0;
    if (e < E)
      for (int v = 0; v < kLossWaves; ++v) s += (double)sums[v][e];
    finish_loss(s, e < E ? cnt[e] : 0, cnt[kWidth], e < E, e, E, K, coef, counts, prob, loss, buf);
  } else {
    float2* out = part + (size_t)blockIdx.x * (E + 1);
    for (int e = threadIdx.x; e < E; e += kLossThreads) {
      float s = 0.f;
      for (int v = 0; v < kLossWaves; ++v) s += sums[v][e];
      out[e] = make_float2(s, __int_as_float(cnt[e]));
    }
    if (threadIdx.x == 0) out[E] = make_float2(0.f, __int_as_float(cnt[kWidth]));
  }
}

// Many blocks' sums to kFold of them: line y adds blocks y, y + kFold, ...
// They go on as f32, half a step of 2^-24 each, as the blocks' own sums are:
// the last kernel reads one format whether they were folded or not.
constexpr int kFold = 16;
__global__ __launch_bounds__(kWave) void balance_fold_kernel(const float2* __restrict__ part,
                                                             int nblk, int E,
                                                             float2* __restrict__ out) {
  const int e = blockIdx.x * kWave + threadIdx.x;
  if (e > E) return;
  double s = 0.0;
  int32_t c = 0;
#pragma unroll 8
  for (int b = blockIdx.y; b < nblk; b += kFold) {
    const float2 v = part[(size_t)b * (E + 1) + e];
    s += (double)v.x;
    c += __float_as_int(v.y);
  }
  out[(size_t)blockIdx.y * (E + 1) + e] = make_float2((float)s, __int_as_float(c));
}

// One block: the blocks' sums in order, the means, and the loss. `ways`
// threads an expert (of Ep >= E + 1, the last one for the valid tokens), each
// over every ways-th block, eight loads in flight.
__global__ __launch_bounds__(kLossThreads) void balance_final_kernel(
    const float2* __restrict__ part, int nblk, int E, int K, int ways, float coef,
    int32_t* __restrict__ counts, float* __restrict__ prob, float* __restrict__ loss) {
  __shared__ double buf[kLossThreads];
  __shared__ int32_t sc[kLossThreads];
  __shared__ int32_t n_all;
  const int tid = threadIdx.x;
  const int Ep = kLossThreads / ways;
  const int way = tid / Ep;
  // experts e, e + Ep, ...: more than one only where E + 1 > 1024
  double s = 0.0;
  int32_t c = 0;
  const int e = tid % Ep;
  auto walk = [&](int e_) {
    s = 0.0;
    c = 0;
    constexpr int kDeep = 8;
    for (int b0 = way; b0 < nblk; b0 += ways * kDeep) {
      float2 v[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int b = b0 + u * ways;
        v[u] = b < nblk ? part[(size_t)b * (E + 1) + e_] : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        s += (double)v[u].x;
        c += __float_as_int(v[u].y);
      }
    }
  };
  if (E + 1 > Ep) {  // E = 1024: the valid tokens first, by the first thread
    if (tid == 0) {
      walk(E);
      n_all = c;
    }
    __syncthreads();
  }
  if (e <= E) walk(e);
  buf[tid] = s;
  sc[tid] = c;
  __syncthreads();
  if (way == 0) {
    for (int w = 1; w < ways; ++w) {
      s += buf[w * Ep + e];
      c += sc[w * Ep + e];
    }
    if (e == E) n_all = c;
  }
  __syncthreads();
  finish_loss(s, c, n_all, way == 0 && e < E, e, E, K, coef, counts, prob, loss, buf);
}

template <int L, int EPL, bool VEC>
__global__ __launch_bounds__(kGradThreads) void route_backward_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, const uint8_t* __restrict__ token_mask,
    const int32_t* __restrict__ counts, const float* __restrict__ dloss, int T, int E, int K,
    int renorm, float coef, float* __restrict__ dlogits) {
  constexpr int kGroups = kGradThreads / L;
  // The selected experts' terms of each lane group's token, else zeros. Only
  // the group's own wave uses its row, and a wave's LDS accesses run in
  // order. An expert that a token holds twice is added to twice by one
  // instruction: the sum is the same either way round. Three times and more
  // the lanes' order counts, which the hardware keeps from run to run (seen
  // with experts held up to 32 times, not promised by a document).
  __shared__ __align__(16) float picked[kGroups][L * EPL];
  const int q = threadIdx.x & (L - 1);
  const int grp = threadIdx.x / L;
#pragma unroll
  for (int j = 0; j < EPL; ++j) picked[grp][expert_of<L, EPL, VEC>(q, j)] = 0.f;
  wave_lds_fence();
  float f[EPL], c = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) f[j] = 0.f;
  if (counts != nullptr) {
    const int n = counts[E];
    const float share = n > 0 ? 1.0f / ((float)n * (float)K) : 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = expert_of<L, EPL, VEC>(q, j);
      if (e < E) f[j] = (float)counts[e] * share;
    }
    c = (dloss != nullptr ? *dloss : 1.0f) * coef * (float)E * share * (float)K;
  }
  // the same rounds for every lane of a block
  for (uint32_t t0 = blockIdx.x * kGroups; t0 < (uint32_t)T; t0 += gridDim.x * kGroups) {
    const uint32_t t = t0 + grp;
    const bool inside = t < (uint32_t)T;
    const bool live = inside && (token_mask == nullptr || token_mask[t] != 0);
    const float* row = logits + (size_t)(live ? t : 0) * E;
    float p[EPL], shift, denom;
    load_token<L, EPL, VEC>(row, E, q, live, p);
    int id = -1;
    float z = -INFINITY, up = 0.f;
    if (dw != nullptr && live && q < K) {
      const int v = ids[(size_t)t * K + q];
      if (v >= 0 && v < E) {
        id = v;
        z = row[v];
        up = dw[(size_t)t * K + q];
      }
    }
    token_softmax<L, EPL>(p, &shift, &denom);
    float d[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) d[j] = 0.f;
    if (dw != nullptr) {
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
      if (id >= 0) atomicAdd(&picked[grp][id], mine);
      wave_lds_fence();
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        float* at = &picked[grp][expert_of<L, EPL, VEC>(q, j)];
        d[j] += *at;
        *at = 0.f;
      }
      wave_lds_fence();
    }
    if (counts != nullptr) {
      float part = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) part = fmaf(f[j], p[j], part);
      const float mean = lanes_sum<L>(part);
#pragma unroll
      for (int j = 0; j < EPL; ++j) d[j] = fmaf(c * p[j], f[j] - mean, d[j]);
    }
    if (inside) {
      float* out = dlogits + (size_t)t * E;
#pragma unroll
      for (int j = 0; j < EPL; ++j) d[j] = live ? d[j] : 0.f;
      if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < EPL; j += 4) {
          const int e = expert_of<L, EPL, VEC>(q, j);
          if (e < E)
            *reinterpret_cast<float4*>(out + e) = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const int e = expert_of<L, EPL, VEC>(q, j);
          if (e < E) out[e] = d[j];
        }
      }
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

// f(lanes, logits a lane, vectors): vectors where rows are whole aligned
// 16-byte vectors and a lane holds one at least.
template <typename F>
void with_lanes(int E, int K, bool aligned, F&& f) {
  using std::integral_constant;
  const int L = lanes_for(E, K);
  const int epl = ceil_div(E, L);
  const bool vec = aligned && E % 4 == 0 && epl > 2;
  auto pick = [&](auto l) {
    if (epl <= 1)
      f(l, integral_constant<int, 1>{}, std::false_type{});
    else if (epl <= 2)
      f(l, integral_constant<int, 2>{}, std::false_type{});
    else if (epl <= 4 && vec)
      f(l, integral_constant<int, 4>{}, std::true_type{});
    else if (epl <= 4)
      f(l, integral_constant<int, 4>{}, std::false_type{});
    else if (vec)
      f(l, integral_constant<int, 8>{}, std::true_type{});
    else
      f(l, integral_constant<int, 8>{}, std::false_type{});
  };
  if (L == 8)
    pick(integral_constant<int, 8>{});
  else if (L == 16)
    pick(integral_constant<int, 16>{});
  else if (L == 32)
    pick(integral_constant<int, 32>{});
  else {  // over 256 experts
    auto wide = [&](auto v) {
      if (epl <= 8)
        f(integral_constant<int, kWave>{}, integral_constant<int, 8>{}, v);
      else
        f(integral_constant<int, kWave>{}, integral_constant<int, 16>{}, v);
    };
    if (vec)
      wide(std::true_type{});
    else
      wide(std::false_type{});
  }
}

// Blocks of `per` tokens each; T is up to 2^31 - 1, where T + per - 1 would overflow.
int token_blocks(int T, int per) { return T > 0 ? (T - 1) / per + 1 : 0; }

int balance_blocks(int T, int E, int K) {
  const int rounds = token_blocks(T, kLossThreads / lanes_for(E, K));
  return rounds <= kLossRounds ? 1 : std::min(kMaxBlocks, ceil_div(rounds, 2));
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int K) {
  return ((size_t)balance_blocks(T, E, K) + kFold) * (size_t)(E + 1) * sizeof(float2);
}

moe_status_t launch_balance_loss(const float* logits, const int32_t* ids,
                                 const uint8_t* token_mask, int T, int E, int K, float coef,
                                 int32_t* counts, float* prob, float* loss, void* ws,
                                 hipStream_t stream) {
  int nblk = balance_blocks(T, E, K);
  float2* part = static_cast<float2*>(ws);
  with_lanes(E, K, aligned16(logits), [&](auto l, auto epl, auto vec) {
    constexpr int L = decltype(l)::value, EPL = decltype(epl)::value;
    if (nblk == 1)
      balance_partial_kernel<L, EPL, decltype(vec)::value, true><<<1, kLossThreads, 0, stream>>>(
          logits, ids, token_mask, T, E, K, nullptr, coef, counts, prob, loss);
    else
      balance_partial_kernel<L, EPL, decltype(vec)::value, false>
          <<<nblk, kLossThreads, 0, stream>>>(logits, ids, token_mask, T, E, K, part, coef,
                                              counts, prob, loss);
  });
  if (nblk > 1) {
    // one block reads the sums of many at the rate of one compute unit (256 blocks of 256
    // experts: 38 us)
    if (nblk > 2 * kFold) {
      float2* folded = part + (size_t)nblk * (E + 1);
      balance_fold_kernel<<<dim3(ceil_div(E + 1, kWave), kFold), kWave, 0, stream>>>(part, nblk,
                                                                                     E, folded);
      part = folded;
      nblk = kFold;
    }
    int ways = 1;
    while (2 * ways * (E + 1) <= kLossThreads) ways *= 2;
    balance_final_kernel<<<1, kLossThreads, 0, stream>>>(part, nblk, E, K, ways, coef, counts,
                                                         prob, loss);
  }
  return launch_status();
}

moe_status_t launch_route_backward(const float* logits, const int32_t* ids, const float* dw,
                                   const uint8_t* token_mask, const int32_t* counts,
                                   const float* dloss, int T, int E, int K, int renorm,
                                   float coef, float* dlogits, hipStream_t stream) {
  if (T == 0) return MOE_OK;
  with_lanes(E, K, aligned16(logits) && aligned16(dlogits), [&](auto l, auto epl, auto vec) {
    constexpr int L = decltype(l)::value;
    const int blocks = std::min(token_blocks(T, kGradThreads / L), kGradBlocks);
    route_backward_kernel<L, decltype(epl)::value, decltype(vec)::value>
        <<<blocks, kGradThreads, 0, stream>>>(logits, ids, dw, token_mask, counts, dloss, T, E,
                                              K, renorm, coef, dlogits);
  });
  return launch_status();
}

}  // namespace moe
