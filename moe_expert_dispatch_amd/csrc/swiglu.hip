// The SwiGLU of the gate/up product's output, for a forward pass that keeps
// that output for its gradient (moe_grouped_gemm fuses the two and keeps only
// the result):  act[r, j] = silu(h[r, j]) * h[r, I + j],  h [rows, 2I].
//
// Bound by the bytes, three values of the row's type for each result. A block
// takes 512 consecutive vectors of 8 results, whatever the rows' width, a thread
// two of them with both loads in flight: 32768 rows of 1024 bf16 in 47 to 49 us, 4.2
// TB/s (62 us with a vector a thread and a full division).
#include "common.h"
#include "vec8.h"

namespace moe {
namespace {

constexpr int kSwigluThreads = 256, kSwigluVec = 2;

// silu(g) u. For bf16 results the quotient's and the exponential's fast forms,
// as in the fused product: their few 2^-24 are far below the rounding.
__device__ __forceinline__ float gate(float g, float u, const uint16_t*) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}
__device__ __forceinline__ float gate(float g, float u, const float*) {
  return g / (1.0f + expf(-g)) * u;
}

template <typename XT>
__global__ __launch_bounds__(kSwigluThreads) void swiglu_kernel(const XT* __restrict__ h,
                                                                const int32_t* __restrict__ offsets,
                                                                int S, int max_rows, int I,
                                                                XT* __restrict__ act) {
  const uint32_t nvec = (uint32_t)I / 8u;
  const size_t first = (size_t)max(0, offsets[0]), rows = (size_t)max(0, min(offsets[S], max_rows));
  const uint64_t start = (uint64_t)folded_block() * (kSwigluThreads * kSwigluVec);
  const uint64_t row0 = start / nvec;
  const uint32_t rest = (uint32_t)(start - row0 * nvec);
  typedef decltype(raw8(h)) Raw;
  Raw g[kSwigluVec] = {}, u[kSwigluVec] = {};
  size_t row[kSwigluVec];
  uint32_t col[kSwigluVec];
#pragma unroll
  for (int k = 0; k < kSwigluVec; ++k) {
    const uint32_t q = rest + threadIdx.x + k * kSwigluThreads;
    const uint32_t down = q / nvec;
    row[k] = (size_t)row0 + down;
    col[k] = (q - down * nvec) * 8u;
    if (row[k] >= first && row[k] < rows) {
      g[k] = raw8(h + row[k] * 2 * I + col[k]);
      u[k] = raw8(h + row[k] * 2 * I + I + col[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kSwigluVec; ++k) {
    if (row[k] < first || row[k] >= rows) continue;
    float a[8], b[8];
    unpack8(g[k], a);
    unpack8(u[k], b);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = gate(a[i], b[i], h);
    store8(act + row[k] * I + col[k], a);
  }
}

}  // namespace

moe_status_t launch_swiglu(const void* h, bool bf16, const int32_t* offsets, int S, int max_rows,
                           int I, void* act, hipStream_t stream) {
  if (max_rows == 0) return MOE_OK;
  const int64_t vecs = (int64_t)max_rows * (I / 8);
  const int per = kSwigluThreads * kSwigluVec;
  const dim3 grid = folded((vecs + per - 1) / per, kSwigluThreads);
  if (bf16)
    swiglu_kernel<uint16_t><<<grid, kSwigluThreads, 0, stream>>>(
        static_cast<const uint16_t*>(h), offsets, S, max_rows, I, static_cast<uint16_t*>(act));
  else
    swiglu_kernel<float><<<grid, kSwigluThreads, 0, stream>>>(
        static_cast<const float*>(h), offsets, S, max_rows, I, static_cast<float*>(act));
  return launch_status();
}

}  // namespace moe
