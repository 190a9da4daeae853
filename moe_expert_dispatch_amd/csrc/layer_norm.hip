// Layer norm with the residual's addition, and an output in E4M3 codes for
// the FP8 experts.
//
//   h = x + residual (f32), residual_out = round(h)
//   v = (h - mean h) / sqrt(mean (h - mean h)^2 + eps) * gamma + beta
//   y = round(v), q = quantize(v, scale)   (the rule of moe_quantize_fp8)
//
// As the root-mean-square norm: a row stays in f32 registers from the load to
// the stores, one vector of 8 values a thread up to rows of 8192. Rows of up
// to 512 values are parts of waves, several to a block, and need no barrier.
#include "norm_row.h"

namespace moe {
namespace {

template <typename XT, int VPT, int L>
__global__ __launch_bounds__(L == 0 ? 1024 : kNormGroupThreads) void layer_norm_kernel(
    const XT* x, const XT* residual, const XT* __restrict__ gamma, const XT* __restrict__ beta,
    int T, int H, float eps, XT* residual_out, XT* y, uint8_t* __restrict__ q, float inv) {
  __shared__ RowParts part;
  constexpr bool kGuess = L == 0 && VPT == 1;
  constexpr int kRows = L == 0 ? 1 : kNormGroupThreads / (L == 0 ? 1 : L);
  const int64_t t = (int64_t)folded_block() * kRows + (L == 0 ? 0 : threadIdx.x / (L == 0 ? 1 : L));
  if (t >= T) return;
  const int first = L == 0 ? threadIdx.x : threadIdx.x % (L == 0 ? 1 : L);
  const int stride = L == 0 ? blockDim.x : L;
  const int nvec = H / 8;
  const size_t row = (size_t)t * H;
  float h[VPT][8] = {};
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = first + j * stride;
    if (v < nvec) {
      load8(x + row + v * 8, h[j]);
      if (residual != nullptr) {
        float r[8];
        load8(residual + row + v * 8, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] += r[i];
      }
      if (!kGuess && residual_out != nullptr) store8(residual_out + row + v * 8, h[j]);
    }
  }
  float guess = 0.f, keep[8] = {};
  if constexpr (kGuess) {
    float v[8], r[8] = {};
    load8(x + row, v);
    if (residual != nullptr) load8(residual + row, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] += r[i];
      keep[i] = h[0][i];
    }
    guess = mean8(v);
  }
  normalize_row<true, VPT, L>(h, first, stride, nvec, H, eps, part, guess);
  // behind the first barrier: residual_out may be x or the residual, whose first
  // values every thread reads
  if constexpr (kGuess)
    if (first < nvec && residual_out != nullptr) store8(residual_out + row + first * 8, keep);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = first + j * stride;
    if (v < nvec) {
      float g[8], b[8] = {};
      load8(gamma + v * 8, g);
      if (beta != nullptr) load8(beta + v * 8, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = fmaf(h[j][i], g[i], b[i]);
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

template <typename XT, int VPT, int L>
void launch_v(const void* x, const void* residual, const void* gamma, const void* beta, int T, int H,
              float eps, void* residual_out, void* y, uint8_t* q, float inv, hipStream_t stream) {
  const int threads = L == 0 ? ceil_div(ceil_div(H / 8, VPT), kWave) * kWave : kNormGroupThreads;
  const int rows = L == 0 ? 1 : kNormGroupThreads / (L == 0 ? 1 : L);
  layer_norm_kernel<XT, VPT, L>
      <<<folded(((int64_t)T + rows - 1) / rows, threads), threads, 0, stream>>>(
          static_cast<const XT*>(x), static_cast<const XT*>(residual),
          static_cast<const XT*>(gamma), static_cast<const XT*>(beta), T, H, eps,
          static_cast<XT*>(residual_out), static_cast<XT*>(y), q, inv);
}

template <typename XT>
void launch_typed(const void* x, const void* residual, const void* gamma, const void* beta, int T,
                  int H, float eps, void* residual_out, void* y, uint8_t* q, float inv,
                  hipStream_t stream) {
  const int nvec = H / 8;
  auto go = [&](auto vpt, auto lanes) {
    launch_v<XT, decltype(vpt)::value, decltype(lanes)::value>(
        x, residual, gamma, beta, T, H, eps, residual_out, y, q, inv, stream);
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 0> block;
  switch (norm_lanes(nvec)) {
    case 16: return go(one, std::integral_constant<int, 16>{});
    case 32: return go(one, std::integral_constant<int, 32>{});
    case 64: return go(one, std::integral_constant<int, 64>{});
  }
  if (nvec <= 1024)
    go(one, block);
  else if (nvec <= 2048)
    go(std::integral_constant<int, 2>{}, block);
  else
    go(std::integral_constant<int, 4>{}, block);
}

}  // namespace

moe_status_t launch_layer_norm(const void* x, const void* residual, const void* gamma,
                               const void* beta, bool bf16, int T, int H, float eps,
                               void* residual_out, void* y, uint8_t* q, float scale,
                               hipStream_t stream) {
  if (T == 0) return MOE_OK;
  const float inv = q != nullptr ? 1.0f / scale : 0.0f;
  if (bf16)
    launch_typed<uint16_t>(x, residual, gamma, beta, T, H, eps, residual_out, y, q, inv, stream);
  else
    launch_typed<float>(x, residual, gamma, beta, T, H, eps, residual_out, y, q, inv, stream);
  return launch_status();
}

}  // namespace moe
