// Gradients of the grouped products in f32 (gemm_grad.hip has the formulas and
// the bf16 kernels), on the f32 matrix instructions: v_mfma_f32_32x32x2_f32
// multiplies and adds in f32, 256 operations a cycle and compute unit.
//
// Tiles of 64 x 64, four waves of 32 x 32, slices of 32 contracted values in
// LDS with the contraction outermost, so that a lane's operand is one value
// beside its neighbours' in both products.
#include "grouped_tiles.h"
#include "vec8.h"

namespace moe {
namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int kTile32 = kGradTileF32, kSlice32 = 32, kThreads32 = 256;
constexpr int kPitch = kTile32 + 4;

struct Args32 {
  const float* m_side;  // dc [rows, Kd], or dc [rows, M]
  const float* n_side;  // w [S, Kd, N], or a [rows, N]
  const int32_t* offsets;
  int S, max_rows, M, N, Kd;
  const float* h;
  void* out;
  int out_bf16, accumulate, splits;
};

template <bool WEIGHTS>
__global__ __launch_bounds__(kThreads32) void grouped_grad_f32_kernel(Args32 p) {
  __shared__ float ms[kSlice32][kPitch], ns[kSlice32][kPitch];
  __shared__ int32_t tp[WEIGHTS ? 1 : MOE_MAX_SLOTS + 1];
  __shared__ int32_t scratch[WEIGHTS ? 1 : kThreads32];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int wm = wave >> 1, wn = wave & 1;
  const int NT = ceil_div(p.N, kTile32), MT = WEIGHTS ? ceil_div(p.M, kTile32) : 0;
  int RT = 0;
  if constexpr (!WEIGHTS) {
    tile_prefix<kThreads32, kTile32>(p.offsets, p.S, p.max_rows, tp, scratch);
    RT = tp[p.S];
  }
  const int total = WEIGHTS ? p.S * p.splits * MT * NT : RT * NT;
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int s, m0 = 0, n0, row0, rows, split = 0;
    if constexpr (WEIGHTS) {
      const int z = item / (MT * NT), t = item - z * MT * NT;
      s = z / p.splits;
      split = z - s * p.splits;
      m0 = t / NT * kTile32;
      n0 = t % NT * kTile32;
      int lo, hi;
      slot_rows(p.offsets, s, p.max_rows, &lo, &hi);
      const int each = ceil_div(ceil_div(hi - lo, kSlice32), p.splits) * kSlice32;
      row0 = min(lo + split * each, hi);
      rows = min(hi - row0, each);
    } else {
      const int rt = item / NT;
      n0 = item % NT * kTile32;
      s = tile_slot(tp, p.S, rt);
      int lo, hi;
      slot_rows(p.offsets, s, p.max_rows, &lo, &hi);
      row0 = lo + (rt - tp[s]) * kTile32;
      rows = min(kTile32, hi - row0);
    }
    const int depth = WEIGHTS ? rows : p.Kd;
    // two vectors of 4 of each operand a thread; zeros past the ends
    float4 mv[2], nv[2];
    auto load = [&](int k0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int q = tid + u * kThreads32;
        const int k = k0 + q / 16, c = q % 16 * 4;
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        const float* n = WEIGHTS ? p.n_side + ((size_t)row0 + k) * p.N + n0 + c
                                 : p.n_side + ((size_t)s * p.Kd + k) * p.N + n0 + c;
        nv[u] = k < depth && n0 + c < p.N ? *reinterpret_cast<const float4*>(n) : zero;
        if constexpr (WEIGHTS) {
          mv[u] = k < depth && m0 + c < p.M ? *reinterpret_cast<const float4*>(
                                                  p.m_side + ((size_t)row0 + k) * p.M + m0 + c)
                                            : zero;
        } else {
          const int r = q / 8, kk = k0 + q % 8 * 4;
          mv[u] = r < rows && kk < p.Kd ? *reinterpret_cast<const float4*>(
                                              p.m_side + ((size_t)row0 + r) * p.Kd + kk)
                                        : zero;
        }
      }
    };
    auto store = [&]() {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int q = tid + u * kThreads32;
        *reinterpret_cast<float4*>(&ns[q / 16][q % 16 * 4]) = nv[u];
        if constexpr (WEIGHTS) {
          *reinterpret_cast<float4*>(&ms[q / 16][q % 16 * 4]) = mv[u];
        } else {
          const int r = q / 8, kk = q % 8 * 4;
          ms[kk][r] = mv[u].x;
          ms[kk + 1][r] = mv[u].y;
          ms[kk + 2][r] = mv[u].z;
          ms[kk + 3][r] = mv[u].w;
        }
      }
    };
    floatx16 acc = {};
    if (depth > 0) load(0);
    for (int k0 = 0; k0 < depth; k0 += kSlice32) {
      __syncthreads();  // the slice before has been read
      store();
      __syncthreads();
      if (k0 + kSlice32 < depth) load(k0 + kSlice32);
#pragma unroll
      for (int k = 0; k < kSlice32; k += 2) {
        const float a = ms[k + (lane >> 5)][wm * 32 + (lane & 31)];
        const float b = ns[k + (lane >> 5)][wn * 32 + (lane & 31)];
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(b, a, acc, 0, 0, 0);
      }
    }
    // register v: column 8 (v / 4) + 4 (lane / 32) + v % 4, row lane % 32
    const int r = wm * 32 + (lane & 31);
    if (WEIGHTS ? m0 + r >= p.M : r >= rows) continue;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = n0 + wn * 32 + 8 * g + 4 * (lane >> 5);
      if (col >= p.N) continue;
      float4 o = make_float4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
      if constexpr (WEIGHTS) {
        const size_t at = ((((size_t)split * p.S + s) * p.M) + m0 + r) * p.N + col;
        if (p.out_bf16) {
          uint2* q = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at);
          if (p.accumulate) {
            const uint2 v = *q;
            o.x = bf16_to_f32(v.x & 0xffffu) + o.x;
            o.y = bf16_to_f32(v.x >> 16) + o.y;
            o.z = bf16_to_f32(v.y & 0xffffu) + o.z;
            o.w = bf16_to_f32(v.y >> 16) + o.w;
          }
          *q = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        } else {
          float4* q = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
          if (p.accumulate) {
            const float4 v = *q;
            o.x = v.x + o.x; o.y = v.y + o.y; o.z = v.z + o.z; o.w = v.w + o.w;
          }
          *q = o;
        }
      } else if (p.h != nullptr) {
        const size_t at = ((size_t)row0 + r) * 2 * p.N + col;
        const float4 g4 = *reinterpret_cast<const float4*>(p.h + at);
        const float4 u4 = *reinterpret_cast<const float4*>(p.h + at + p.N);
        float d[4] = {o.x, o.y, o.z, o.w}, gt[4] = {g4.x, g4.y, g4.z, g4.w},
              u[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float sg = 1.0f / (1.0f + expf(-gt[v]));
          const float silu = gt[v] * sg;
          gt[v] = d[v] * u[v] * (sg + silu * (1.0f - sg));
          u[v] = d[v] * silu;
        }
        float* q = static_cast<float*>(p.out) + at;
        *reinterpret_cast<float4*>(q) = make_float4(gt[0], gt[1], gt[2], gt[3]);
        *reinterpret_cast<float4*>(q + p.N) = make_float4(u[0], u[1], u[2], u[3]);
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + ((size_t)row0 + r) * p.N + col) = o;
      }
    }
  }
}

int grid32(int64_t items) {
  const int64_t most = 4 * (int64_t)device_cu_count();
  return items < most ? (int)items : (int)most;
}

// out[i] = (accumulate: out[i] +) the sum over the splits of part[split][i], 8 values a thread.
template <typename OT>
__global__ __launch_bounds__(256) void fold_splits_kernel(const float* __restrict__ part, int splits,
                                                          size_t n, OT* __restrict__ out,
                                                          int accumulate) {
  const size_t i = ((size_t)folded_block() * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  float s[8];
  load8(part + i, s);
  for (int k = 1; k < splits; ++k) {
    float v[8];
    load8(part + (size_t)k * n + i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += v[j];
  }
  if (accumulate) {
    float v[8];
    load8(out + i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = v[j] + s[j];
  }
  store8(out + i, s);
}

}  // namespace

moe_status_t launch_fold_splits(const float* part, int splits, size_t n, void* out, bool out_f32,
                                int accumulate, hipStream_t stream) {
  const dim3 grid = folded((int64_t)((n / 8 + 255) / 256), 256);
  if (out_f32)
    fold_splits_kernel<float><<<grid, 256, 0, stream>>>(part, splits, n, static_cast<float*>(out),
                                                        accumulate);
  else
    fold_splits_kernel<uint16_t><<<grid, 256, 0, stream>>>(part, splits, n,
                                                           static_cast<uint16_t*>(out), accumulate);
  return launch_status();
}

moe_status_t launch_gemm_backward_f32(const void* dc, const int32_t* offsets, int S, int max_rows,
                                      const void* w, int Kd, int N, const void* h, void* out,
                                      hipStream_t stream) {
  Args32 p{};
  p.m_side = static_cast<const float*>(dc);
  p.n_side = static_cast<const float*>(w);
  p.offsets = offsets;
  p.S = S; p.max_rows = max_rows; p.N = N; p.Kd = Kd; p.splits = 1;
  p.h = static_cast<const float*>(h);
  p.out = out;
  const int64_t items =
      (int64_t)(max_rows / kTile32 + 1 + (S < max_rows ? S : max_rows)) * ceil_div(N, kTile32);
  grouped_grad_f32_kernel<false><<<grid32(items), kThreads32, 0, stream>>>(p);
  return launch_status();
}

moe_status_t launch_gemm_weight_grad_f32(const void* dc, const void* a, const int32_t* offsets,
                                         int S, int max_rows, int M, int N, void* dw, bool dw_f32,
                                         int accumulate, void* ws, hipStream_t stream) {
  Args32 p{};
  p.m_side = static_cast<const float*>(dc);
  p.n_side = static_cast<const float*>(a);
  p.offsets = offsets;
  p.S = S; p.max_rows = max_rows; p.M = M; p.N = N;
  p.splits = grad_splits(S, max_rows, M, N, kTile32);
  p.out = p.splits > 1 ? ws : dw;
  p.out_bf16 = p.splits > 1 ? 0 : !dw_f32;
  p.accumulate = p.splits > 1 ? 0 : accumulate;
  const int64_t items = (int64_t)S * p.splits * ceil_div(M, kTile32) * ceil_div(N, kTile32);
  grouped_grad_f32_kernel<true><<<grid32(items), kThreads32, 0, stream>>>(p);
  if (p.splits > 1)
    return launch_fold_splits(static_cast<const float*>(ws), p.splits, (size_t)S * M * N, dw, dw_f32,
                              accumulate, stream);
  return launch_status();
}

}  // namespace moe
