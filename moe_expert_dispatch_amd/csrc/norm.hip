// Root-mean-square norm with the residual's addition, and an output in E4M3
// codes for the FP8 experts.
//
//   h = x + residual (f32), residual_out = round(h)
//   v = h / sqrt(mean(h^2) + eps) * gamma
//   y = round(v), q = quantize(v, scale)   (the rule of moe_quantize_fp8)
//
// One block per row. Every thread keeps its VPT vectors of 8 values in f32
// registers from the load to the stores, so the row is read once and both
// outputs come from the unrounded v. The sum of squares is f32: per thread,
// then per wave, then over the waves in order, so it does not depend on
// scheduling. A row whose squares leave f32's range is summed again in f64.
//
// Bound by the bytes: 8192 rows of 5120 bf16 with residual and codes 71 us,
// 5.3 TB/s; 16384 of 4096 103 us, 5.9 TB/s. One vector a thread (VPT = 1) is
// the fastest wherever 1024 threads hold a row: with two a thread 72 and 111
// us, with four 79 and 121. A single row of 4096 takes 2.4 us. Rows of 512 and
// 1024 run at 6.5 TB/s and more (134 and 268 MB, in part in the memory-side
// cache); shorter ones leave lanes of their one wave idle: 524288 rows of 128
// (the norm of heads) 115 us, 2.3 TB/s.
#include "common.h"
#include "vec8.h"

namespace moe {
namespace {

// Below this mean (eps included) squares may have lost bits that count to
// f32's least number: here the halves of 2^-149 lost are 2^-70 of it at most.
constexpr float kLeastMean = 0x1p-80f;

// h / sqrt(mean(h^2) + eps) in place, for a block whose squares leave f32's
// range: the sum and the quotient in f64, where every square of an f32 number
// is exact.
template <int VPT>
__device__ __forceinline__ void normalize_wide(float (&h)[VPT][8], int nvec, int H, float eps) {
  __shared__ double part[16];
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if ((int)(threadIdx.x + j * blockDim.x) < nvec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma((double)h[j][i], (double)h[j][i], ss);
    }
  }
#pragma unroll
  for (int o = kWave / 2; o > 0; o /= 2) ss += __shfl_xor(ss, o, kWave);
  if (lane_id() == 0) part[threadIdx.x / kWave] = ss;
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < (int)(blockDim.x / kWave); ++w) total += part[w];
  const double r = 1.0 / sqrt(total / H + (double)eps);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if ((int)(threadIdx.x + j * blockDim.x) < nvec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = (float)((double)h[j][i] * r);
    }
  }
}

template <typename XT, int VPT>
__global__ __launch_bounds__(1024) void rms_norm_kernel(
    const XT* x, const XT* residual, const XT* __restrict__ gamma, int T, int H, float eps,
    XT* residual_out, XT* y, uint8_t* __restrict__ q, float inv) {
  __shared__ float part[16];
  if (folded_block() >= (uint32_t)T) return;
  const int nvec = H / 8;
  const size_t row = (size_t)folded_block() * H;
  float h[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    if (v < nvec) {
      load8(x + row + v * 8, h[j]);
      if (residual != nullptr) {
        float r[8];
        load8(residual + row + v * 8, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
    }
  }
  ss = wave_sum(ss);
  if (lane_id() == 0) part[threadIdx.x / kWave] = ss;
  __syncthreads();
  float total = 0.f;
  for (int w = 0; w < (int)(blockDim.x / kWave); ++w) total += part[w];
  const float mean = total / (float)H + eps;
  float r = 1.0f / sqrtf(mean);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    if (v < nvec && residual_out != nullptr) store8(residual_out + row + v * 8, h[j]);
  }
  // the same for the whole block; false for a NaN too
  if (!(mean >= kLeastMean && total < INFINITY)) {
    normalize_wide<VPT>(h, nvec, H, eps);
    r = 1.0f;
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    if (v < nvec) {
      float g[8];
      load8(gamma + v * 8, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = h[j][i] * r * g[i];
      if (y != nullptr) store8(y + row + v * 8, g);
      if (q != nullptr) {
        uint2 c;
        c.x = fp8_q4(g[0], g[1], g[2], g[3], inv);
        c.y = fp8_q4(g[4], g[5], g[6], g[7], inv);
        *reinterpret_cast<uint2*>(q + row + v * 8) = c;
      }
    }
  }
}

template <typename XT, int VPT>
void launch_v(const void* x, const void* residual, const void* gamma, int T, int H, float eps,
              void* residual_out, void* y, uint8_t* q, float inv, hipStream_t stream) {
  const int threads = ceil_div(ceil_div(H / 8, VPT), kWave) * kWave;
  rms_norm_kernel<XT, VPT><<<folded(T, threads), threads, 0, stream>>>(
      static_cast<const XT*>(x), static_cast<const XT*>(residual),
      static_cast<const XT*>(gamma), T, H, eps, static_cast<XT*>(residual_out),
      static_cast<XT*>(y), q, inv);
}

template <typename XT>
void launch_typed(const void* x, const void* residual, const void* gamma, int T, int H,
                  float eps, void* residual_out, void* y, uint8_t* q, float inv,
                  hipStream_t stream) {
  const int nvec = H / 8;
  if (nvec <= 1024)
    launch_v<XT, 1>(x, residual, gamma, T, H, eps, residual_out, y, q, inv, stream);
  else if (nvec <= 2048)
    launch_v<XT, 2>(x, residual, gamma, T, H, eps, residual_out, y, q, inv, stream);
  else
    launch_v<XT, 4>(x, residual, gamma, T, H, eps, residual_out, y, q, inv, stream);
}

}  // namespace

moe_status_t launch_rms_norm(const void* x, const void* residual, const void* gamma, bool bf16,
                             int T, int H, float eps, void* residual_out, void* y, uint8_t* q,
                             float scale, hipStream_t stream) {
  if (T == 0) return MOE_OK;
  const float inv = q != nullptr ? 1.0f / scale : 0.0f;
  if (bf16)
    launch_typed<uint16_t>(x, residual, gamma, T, H, eps, residual_out, y, q, inv, stream);
  else
    launch_typed<float>(x, residual, gamma, T, H, eps, residual_out, y, q, inv, stream);
  return launch_status();
}

}  // namespace moe
