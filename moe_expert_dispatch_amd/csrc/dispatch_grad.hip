// Gradients of the weighted sum back into token order (moe_combine) and of the
// permutation that applies the weights (moe_permute_scaled).
//
//   combine:  out[t] = sum_k w[t,k] y[row(t,k)]
//             dy[row] = round(w[t,k] dout[t]),  dw[t,k] = <dout[t], y[row]>
//   permute:  xp[row] = w[t,k] x[t]
//             dx[t] = sum_k w[t,k] dxp[row],    dw[t,k] = <x[t], dxp[row]>
//
// One block per token, as the combine: the token's row once, its K rows with
// their loads in flight (8 or 4 at a time), dot products in f32 per thread, per
// wave, then over the waves in order. Each output is written by one thread.
//
// Bound by the bytes, 2 P + T rows and P + 2 T: 16384 tokens of 4096 bf16, top-8,
// 415 to 437 us at 5.2 to 5.5 TB/s and 202 at 6.6; 4096 of 2048 58 us (4.9) and 30 (5.6); 64
// tokens of 2048, top-4, 4.4 us.
#include <algorithm>

#include "common.h"
#include "vec8.h"

namespace moe {
namespace {

using moe::load8;  // beside the forms below that go through a resource
using moe::store8;

typedef int int32x4_t __attribute__((ext_vector_type(4)));
constexpr int kNonTemporal = 2;  // rows that one kernel reads or writes once

// Over one row, empty for a pair without one: its loads give zeros, its
// stores are dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* row, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(row), (short)0, (int)bytes,
                                           0x00020000);
}

__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t r, uint32_t off, const uint16_t*,
                                      float* v) {
  const int32x4_t q = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, kNonTemporal);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32((uint32_t)q[i] & 0xffffu);
    v[2 * i + 1] = bf16_to_f32((uint32_t)q[i] >> 16);
  }
}

__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t r, uint32_t off, const float*,
                                      float* v) {
  const int32x4_t a = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, kNonTemporal);
  const int32x4_t b = __builtin_amdgcn_raw_buffer_load_b128(r, (int)(off + 16u), 0, kNonTemporal);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __int_as_float(a[i]);
    v[4 + i] = __int_as_float(b[i]);
  }
}

__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, uint32_t off, const uint16_t*,
                                       const float* v) {
  int32x4_t q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = (int)pack_bf16x2(v[2 * i], v[2 * i + 1]);
  __builtin_amdgcn_raw_buffer_store_b128(q, r, (int)off, 0, kNonTemporal);
}

__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, uint32_t off, const float*,
                                       const float* v) {
  int32x4_t a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __float_as_int(v[i]);
    b[i] = __float_as_int(v[4 + i]);
  }
  __builtin_amdgcn_raw_buffer_store_b128(a, r, (int)off, 0, kNonTemporal);
  __builtin_amdgcn_raw_buffer_store_b128(b, r, (int)(off + 16u), 0, kNonTemporal);
}

constexpr int kThreads = 512;
typedef float Parts[MOE_MAX_TOPK];  // a wave's parts of the token's dot products

// Adds the wave's parts of the dot products of pairs k0 .. k0 + KMAX.
template <int KMAX>
__device__ __forceinline__ void add_dots(const float* dot, int k0, int K, Parts* part) {
#pragma unroll
  for (int kk = 0; kk < KMAX; ++kk) {
    const float s = wave_sum(dot[kk]);
    if (lane_id() == 0 && k0 + kk < K) part[threadIdx.x / kWave][k0 + kk] += s;
  }
}

// The token's rows and weights, and empty parts.
__device__ __forceinline__ void load_pairs(const int32_t* pair_row, const float* w, size_t t, int K,
                                           int32_t* rows, float* wts, Parts* part) {
  if ((int)threadIdx.x < K) {
    rows[threadIdx.x] = pair_row[t * K + threadIdx.x];
    wts[threadIdx.x] = w != nullptr ? w[t * K + threadIdx.x] : 1.0f;
  }
  if (lane_id() < MOE_MAX_TOPK) part[threadIdx.x / kWave][lane_id()] = 0.f;
  __syncthreads();
}

__device__ __forceinline__ void store_dots(const Parts* part, const int32_t* rows, int K,
                                           float* __restrict__ out) {
  __syncthreads();
  if ((int)threadIdx.x < K) {
    float s = 0.f;
    for (int w = 0; w < (int)(blockDim.x / kWave); ++w) s += part[w][threadIdx.x];
    out[threadIdx.x] = rows[threadIdx.x] >= 0 ? s : 0.f;
  }
}

template <typename DT, typename YT, int KMAX, int VEC>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const DT* __restrict__ dout, const YT* __restrict__ y, const int32_t* __restrict__ pair_row,
    const float* __restrict__ w_masked, int T, int K, int H, YT* __restrict__ dy,
    float* __restrict__ dw) {
  const uint32_t t = folded_block();
  if (t >= (uint32_t)T) return;
  __shared__ int32_t rows[MOE_MAX_TOPK];
  __shared__ float wts[MOE_MAX_TOPK];
  __shared__ Parts part[kThreads / kWave];
  load_pairs(pair_row, w_masked, t, K, rows, wts, part);
  const int nvec = H / 8;
  const uint32_t row_bytes = (uint32_t)H * (uint32_t)sizeof(YT);
  const DT* drow = dout + (size_t)t * H;
  for (int v0 = threadIdx.x; v0 - (int)threadIdx.x < nvec; v0 += VEC * blockDim.x) {
    float d[VEC][8] = {};
    uint32_t off[VEC];
#pragma unroll
    for (int u = 0; u < VEC; ++u) {
      const int v = v0 + u * blockDim.x;
      off[u] = v < nvec ? (uint32_t)v * 8u * (uint32_t)sizeof(YT) : row_bytes;
      if (v < nvec) load8(drow + v * 8, d[u]);
    }
    for (int k0 = 0; k0 < K; k0 += KMAX) {
      if (dw != nullptr) {
        float yv[KMAX][VEC][8], dot[KMAX] = {};
#pragma unroll
        for (int kk = 0; kk < KMAX; ++kk) {
          const int r = k0 + kk < K ? rows[k0 + kk] : -1;
          const __amdgpu_buffer_rsrc_t rr =
              row_rsrc(y + (size_t)(r >= 0 ? r : 0) * H, r >= 0 ? row_bytes : 0u);
#pragma unroll
          for (int u = 0; u < VEC; ++u) load8(rr, off[u], y, yv[kk][u]);
        }
#pragma unroll
        for (int kk = 0; kk < KMAX; ++kk)
#pragma unroll
          for (int u = 0; u < VEC; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[kk] = fmaf(d[u][i], yv[kk][u][i], dot[kk]);
        add_dots<KMAX>(dot, k0, K, part);
      }
      if (dy != nullptr) {
#pragma unroll
        for (int kk = 0; kk < KMAX; ++kk) {
          const int r = k0 + kk < K ? rows[k0 + kk] : -1;
          if (r < 0) continue;  // block-uniform
          const float wk = wts[k0 + kk];
          const __amdgpu_buffer_rsrc_t rr = row_rsrc(dy + (size_t)r * H, row_bytes);
#pragma unroll
          for (int u = 0; u < VEC; ++u) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = d[u][i] * wk;
            store8(rr, off[u], y, o);
          }
        }
      }
    }
  }
  if (dw != nullptr) store_dots(part, rows, K, dw + (size_t)t * K);
}

template <typename DT, typename OT, int KMAX, int VEC>
__global__ __launch_bounds__(kThreads) void permute_backward_kernel(
    const DT* __restrict__ dxp, const int32_t* __restrict__ pair_row,
    const float* __restrict__ pair_w, const DT* __restrict__ x, int T, int K, int H,
    OT* __restrict__ dx, int accumulate, float* __restrict__ dw) {
  const uint32_t t = folded_block();
  if (t >= (uint32_t)T) return;
  __shared__ int32_t rows[MOE_MAX_TOPK];
  __shared__ float wts[MOE_MAX_TOPK];
  __shared__ Parts part[kThreads / kWave];
  load_pairs(pair_row, pair_w, t, K, rows, wts, part);
  const int nvec = H / 8;
  const uint32_t row_bytes = (uint32_t)H * (uint32_t)sizeof(DT);
  const DT* xrow = x + (size_t)t * H;
  OT* o = dx + (size_t)t * H;
  for (int v0 = threadIdx.x; v0 - (int)threadIdx.x < nvec; v0 += VEC * blockDim.x) {
    float xv[VEC][8] = {}, acc[VEC][8] = {};
    uint32_t off[VEC];
#pragma unroll
    for (int u = 0; u < VEC; ++u) {
      const int v = v0 + u * blockDim.x;
      off[u] = v < nvec ? (uint32_t)v * 8u * (uint32_t)sizeof(DT) : row_bytes;
      if (v < nvec) load8(xrow + v * 8, xv[u]);
    }
    for (int k0 = 0; k0 < K; k0 += KMAX) {
      float g[KMAX][VEC][8], dot[KMAX] = {};
#pragma unroll
      for (int kk = 0; kk < KMAX; ++kk) {
        const int r = k0 + kk < K ? rows[k0 + kk] : -1;
        const __amdgpu_buffer_rsrc_t rr =
            row_rsrc(dxp + (size_t)(r >= 0 ? r : 0) * H, r >= 0 ? row_bytes : 0u);
#pragma unroll
        for (int u = 0; u < VEC; ++u) load8(rr, off[u], dxp, g[kk][u]);
      }
#pragma unroll
      for (int kk = 0; kk < KMAX; ++kk) {
        if (k0 + kk >= K || rows[k0 + kk] < 0) continue;  // block-uniform
        const float wk = wts[k0 + kk];
#pragma unroll
        for (int u = 0; u < VEC; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[kk] = fmaf(xv[u][i], g[kk][u][i], dot[kk]);
            acc[u][i] = fmaf(wk, g[kk][u][i], acc[u][i]);
          }
      }
      add_dots<KMAX>(dot, k0, K, part);
    }
#pragma unroll
    for (int u = 0; u < VEC; ++u) {
      const int v = v0 + u * blockDim.x;
      if (v >= nvec) continue;
      if (accumulate) {
        float prev[8];
        load8(o + v * 8, prev);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[u][i] = prev[i] + acc[u][i];
      }
      store8(o + v * 8, acc[u]);
    }
  }
  store_dots(part, rows, K, dw + (size_t)t * K);
}

// 32 bytes of each row a thread, whole waves, as many as hold the row up to 512
// threads (2056 values of f32 are 257 vectors: 256 threads would go round twice).
int row_threads(int H, int vec) {
  return std::min(kThreads, std::max(kWave, ceil_div(H / 8, vec * kWave) * kWave));
}

struct B16 { typedef uint16_t type; };
struct F32 { typedef float type; };

}  // namespace

moe_status_t launch_combine_backward(const void* dout, moe_dtype_t dout_dt, const void* y,
                                     moe_dtype_t y_dt, const int32_t* pair_row,
                                     const float* w_masked, int T, int K, int H, void* dy,
                                     float* dw, hipStream_t stream) {
  if (T == 0) return MOE_OK;
  auto go = [&](auto dk, auto yk, auto kmax) {
    typedef typename decltype(dk)::type DT;
    typedef typename decltype(yk)::type YT;
    constexpr int VEC = sizeof(YT) == 4 ? 1 : 2;
    const int threads = row_threads(H, VEC);
    combine_backward_kernel<DT, YT, decltype(kmax)::value, VEC>
        <<<folded(T, threads), threads, 0, stream>>>(
            static_cast<const DT*>(dout), static_cast<const YT*>(y), pair_row, w_masked, T, K, H,
            static_cast<YT*>(dy), dw);
  };
  auto by_k = [&](auto dk, auto yk) {
    if (K <= 4) go(dk, yk, std::integral_constant<int, 4>{});
    else go(dk, yk, std::integral_constant<int, 8>{});
  };
  const bool db = dout_dt == MOE_DTYPE_BF16, yb = y_dt == MOE_DTYPE_BF16;
  if (db && yb) by_k(B16{}, B16{});
  else if (db) by_k(B16{}, F32{});
  else if (yb) by_k(F32{}, B16{});
  else by_k(F32{}, F32{});
  return launch_status();
}

moe_status_t launch_permute_backward(const void* dx_perm, moe_dtype_t dt, const int32_t* pair_row,
                                     const float* pair_w, const void* x, int T, int K, int H,
                                     void* dx, moe_dtype_t dx_dt, int accumulate, float* dpair_w,
                                     hipStream_t stream) {
  if (T == 0) return MOE_OK;
  if (dpair_w == nullptr)  // the sum alone is the combine's
    return launch_combine(dx_perm, dt, pair_row, pair_w, T, K, H, dx, dx_dt, accumulate, stream);
  auto go = [&](auto dk, auto ok) {
    typedef typename decltype(dk)::type DT;
    typedef typename decltype(ok)::type OT;
    constexpr int VEC = sizeof(DT) == 4 ? 1 : 2;
    const int threads = row_threads(H, VEC);
    // four rows in flight whatever K: with eight fewer blocks fit (8192 tokens of
    // 5120, K = 6 121 us against 112, 1999 of 2056 f32, a quarter of 8 rows each 20
    // against 18)
    permute_backward_kernel<DT, OT, 4, VEC>
        <<<folded(T, threads), threads, 0, stream>>>(
            static_cast<const DT*>(dx_perm), pair_row, pair_w, static_cast<const DT*>(x), T, K, H,
            static_cast<OT*>(dx), accumulate, dpair_w);
  };
  const bool db = dt == MOE_DTYPE_BF16, ob = dx_dt == MOE_DTYPE_BF16;
  if (db && ob) go(B16{}, B16{});
  else if (db) go(B16{}, F32{});
  else if (ob) go(F32{}, B16{});
  else go(F32{}, F32{});
  return launch_status();
}

}  // namespace moe
