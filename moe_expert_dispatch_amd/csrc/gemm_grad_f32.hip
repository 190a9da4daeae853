// Gradients of the grouped products in f32 (gemm_grad.hip has the formulas and
// the bf16 kernels), on the f32 matrix instructions: v_mfma_f32_16x16x4_f32
// multiplies and adds in f32, 256 operations a cycle and compute unit.
//
// Four waves in 2 x 2 on a tile of TILE x TILE, fragments of 16 x 16, slices of
// SLICE contracted values through registers into LDS. An operand that is contiguous along the contraction keeps its rows
// there, the others have the contraction outermost; the pitches put the 16 x 4
// values that a wave reads at once on 64 banks.
//
// 114 to 120 TFLOP/s in either direction (16384 rows, 8 slots of 1024 x 1024 or 16 of
// 2048 x 1024) of the 154 of a large library product: an LDS read of 4 bytes a lane
// for each matrix instruction, and one stage with two barriers a slice.
#include "grouped_tiles.h"
#include "vec8.h"

namespace moe {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int int32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads32 = 256;
constexpr uint32_t kOOB = 0x80000000u;  // past every resource here

// Large tiles for throughput; small ones, with a long slice, where there are
// few: a fragment's chain of products is what takes the time then.
template <int TILE_, int SLICE_>
struct Shape32 {
  static constexpr int TILE = TILE_, SLICE = SLICE_;
};
typedef Shape32<kGradTileF32, 64> Large32;
typedef Shape32<32, 128> Small32;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = (uint32_t)uniform_i32((int)(uint32_t)a);
  const uint32_t hi = (uint32_t)uniform_i32((int)(uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<void*>(((uint64_t)hi << 32) | lo), (short)0,
      uniform_i32((int)bytes), 0x00020000);
}

struct Args32 {
  const float* m_side;  // dc [rows, Kd], or dc [rows, M]
  const float* n_side;  // w [S, Kd, N], or a [rows, N]
  const int32_t* offsets;
  int S, max_rows, M, N, Kd;
  const float* h;
  void* out;
  int out_bf16, accumulate, splits;
};

template <bool WEIGHTS, typename SH>
__global__ __launch_bounds__(kThreads32) void grouped_grad_f32_kernel(Args32 p) {
  constexpr int TILE = SH::TILE, SLICE = SH::SLICE, FR = TILE / 32;
  constexpr int kVec = TILE * SLICE / 4 / kThreads32;  // vectors of 4 of an operand, a thread
  constexpr int kPitchT = TILE + 16, kPitchK = SLICE + 4;
  __shared__ float4 m_part[(WEIGHTS ? SLICE * kPitchT : TILE * kPitchK) / 4];
  __shared__ float4 n_part[SLICE * kPitchT / 4];
  __shared__ int32_t tp[WEIGHTS ? 1 : MOE_MAX_SLOTS + 1];
  __shared__ int32_t scratch[WEIGHTS ? 1 : kThreads32];
  const float* ms = reinterpret_cast<const float*>(m_part);
  const float* ns = reinterpret_cast<const float*>(n_part);
  const int tid = threadIdx.x, lane = lane_id(), wave = uniform_i32(tid / kWave);
  const int wm = wave >> 1, wn = wave & 1;
  const int NT = ceil_div(p.N, TILE), MT = WEIGHTS ? ceil_div(p.M, TILE) : 0;
  int RT = 0;
  if constexpr (!WEIGHTS) {
    tile_prefix<kThreads32, TILE>(p.offsets, p.S, p.max_rows, tp, scratch);
    RT = uniform_i32(tp[p.S]);
  }
  const uint32_t m_row = (uint32_t)(WEIGHTS ? p.M : p.Kd) * 4u, n_row = (uint32_t)p.N * 4u;
  const int total = WEIGHTS ? p.S * p.splits * MT * NT : RT * NT;
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int s, m0 = 0, n0, row0, rows, split = 0, lo, hi;
    if constexpr (WEIGHTS) {
      const int z = item / (MT * NT), t = item - z * MT * NT;
      s = z / p.splits;
      split = z - s * p.splits;
      m0 = t / NT * TILE;
      n0 = t % NT * TILE;
      slot_rows(p.offsets, s, p.max_rows, &lo, &hi);
      split_rows(lo, hi, SLICE, p.splits, split, &row0, &rows);
    } else {
      const int rt = item / NT;
      n0 = item % NT * TILE;
      s = uniform_i32(tile_slot(tp, p.S, rt));
      slot_rows(p.offsets, s, p.max_rows, &lo, &hi);
      row0 = lo + (rt - tp[s]) * TILE;
      rows = min(TILE, hi - row0);
    }
    row0 = uniform_i32(row0);
    rows = uniform_i32(rows);
    const int depth = WEIGHTS ? rows : p.Kd;
    int32x4_t mv[kVec], nv[kVec];
    auto load = [&](int k0) {  // zeros past the ends
      const int left = min(depth - k0, SLICE);
      const __amdgpu_buffer_rsrc_t rm =
          WEIGHTS ? make_rsrc(p.m_side + ((size_t)row0 + k0) * p.M, (uint32_t)left * m_row)
                  : make_rsrc(p.m_side + (size_t)row0 * p.Kd, (uint32_t)rows * m_row);
      const __amdgpu_buffer_rsrc_t rn =
          make_rsrc(WEIGHTS ? p.n_side + ((size_t)row0 + k0) * p.N
                            : p.n_side + ((size_t)s * p.Kd + k0) * p.N,
                    (uint32_t)left * n_row);
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        const int q = tid + u * kThreads32;
        const int k = q / (TILE / 4), c = q % (TILE / 4) * 4;
        nv[u] = __builtin_amdgcn_raw_buffer_load_b128(
            rn, n0 + c < p.N ? (uint32_t)k * n_row + (uint32_t)(n0 + c) * 4u : kOOB, 0, 0);
        if constexpr (WEIGHTS) {
          mv[u] = __builtin_amdgcn_raw_buffer_load_b128(
              rm, m0 + c < p.M ? (uint32_t)k * m_row + (uint32_t)(m0 + c) * 4u : kOOB, 0, 0);
        } else {
          const int r = q / (SLICE / 4), kk = k0 + q % (SLICE / 4) * 4;
          mv[u] = __builtin_amdgcn_raw_buffer_load_b128(
              rm, kk < p.Kd ? (uint32_t)r * m_row + (uint32_t)kk * 4u : kOOB, 0, 0);
        }
      }
    };
    auto store = [&]() {
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        const int q = tid + u * kThreads32;
        const int k = q / (TILE / 4), c = q % (TILE / 4);
        n_part[k * (kPitchT / 4) + c] = __builtin_bit_cast(float4, nv[u]);
        if constexpr (WEIGHTS)
          m_part[k * (kPitchT / 4) + c] = __builtin_bit_cast(float4, mv[u]);
        else
          m_part[q / (SLICE / 4) * (kPitchK / 4) + q % (SLICE / 4)] =
              __builtin_bit_cast(float4, mv[u]);
      }
    };
    // acc[j][i]: 16 columns j by 16 rows i of the wave
    floatx4 acc[FR][FR] = {};
    const int mr = wm * (TILE / 2) + (lane & 15), nc = wn * (TILE / 2) + (lane & 15), kl = lane >> 4;
    if (depth > 0) load(0);
    for (int k0 = 0; k0 < depth; k0 += SLICE) {
      __syncthreads();  // the slice before has been read
      store();
      __syncthreads();
      if (k0 + SLICE < depth) load(k0 + SLICE);
      const int steps = min(SLICE, depth - k0);  // what lies behind is zeros
#pragma unroll 8
      for (int k = 0; k < steps; k += 4) {
        float a[FR], b[FR];
#pragma unroll
        for (int f = 0; f < FR; ++f) {
          a[f] = WEIGHTS ? ms[(k + kl) * kPitchT + mr + f * 16] : ms[(mr + f * 16) * kPitchK + k + kl];
          b[f] = ns[(k + kl) * kPitchT + nc + f * 16];
        }
#pragma unroll
        for (int j = 0; j < FR; ++j)
#pragma unroll
          for (int i = 0; i < FR; ++i)
            acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[j], a[i], acc[j][i], 0, 0, 0);
      }
    }
    // register v of acc[j][i]: column 4 (lane / 16) + v, row lane % 16
#pragma unroll
    for (int i = 0; i < FR; ++i) {
      const int r = mr + i * 16;
      if (WEIGHTS ? m0 + r >= p.M : r >= rows) continue;
#pragma unroll
      for (int j = 0; j < FR; ++j) {
        const int col = n0 + wn * (TILE / 2) + j * 16 + 4 * kl;
        if (col >= p.N) continue;
        float o[4] = {acc[j][i][0], acc[j][i][1], acc[j][i][2], acc[j][i][3]};
        if constexpr (WEIGHTS) {
          const size_t at = ((((size_t)split * p.S + s) * p.M) + m0 + r) * p.N + col;
          if (p.out_bf16) {
            uint2* q = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at);
            if (p.accumulate) {
              const uint2 v = *q;
              o[0] = bf16_to_f32(v.x & 0xffffu) + o[0];
              o[1] = bf16_to_f32(v.x >> 16) + o[1];
              o[2] = bf16_to_f32(v.y & 0xffffu) + o[2];
              o[3] = bf16_to_f32(v.y >> 16) + o[3];
            }
            *q = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
          } else {
            float4* q = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
            if (p.accumulate) {
              const float4 v = *q;
              o[0] = v.x + o[0];
              o[1] = v.y + o[1];
              o[2] = v.z + o[2];
              o[3] = v.w + o[3];
            }
            *q = make_float4(o[0], o[1], o[2], o[3]);
          }
        } else if (p.h != nullptr) {
          const size_t at = ((size_t)row0 + r) * 2 * p.N + col;
          const float4 g4 = *reinterpret_cast<const float4*>(p.h + at);
          const float4 u4 = *reinterpret_cast<const float4*>(p.h + at + p.N);
          float gt[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float sg = 1.0f / (1.0f + expf(-gt[v]));
            const float silu = gt[v] * sg;
            gt[v] = o[v] * u[v] * (sg + silu * (1.0f - sg));
            u[v] = o[v] * silu;
          }
          float* q = static_cast<float*>(p.out) + at;
          *reinterpret_cast<float4*>(q) = make_float4(gt[0], gt[1], gt[2], gt[3]);
          *reinterpret_cast<float4*>(q + p.N) = make_float4(u[0], u[1], u[2], u[3]);
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + ((size_t)row0 + r) * p.N + col) =
              make_float4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
}

// Small tiles up to three large ones for every two compute units. Both sides, small
// and large: rows' gradient of 51 large tiles (8 slots of 83 rows, 264 x 136) 7.9
// and 13.6 us, 324 (16 of 256, 512 x 256) 26.5 and 29.5, 576 42 and 40, 2308 143
// and 109 (79 TFLOP/s); weights' gradient of 120 tiles 4.6 and 5.5, 512 14 and 10,
// 2048 129 and 82 (105 TFLOP/s).
constexpr int kFewTiles = 3, kFewUnits = 2;

int grid32(int64_t items) {
  const int64_t most = 3 * (int64_t)device_cu_count();  // as many as the LDS holds
  return items < most ? (int)items : (int)most;
}

bool few_tiles(int64_t large) { return kFewUnits * large < kFewTiles * (int64_t)device_cu_count(); }

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
  auto go = [&](auto shape) {
    typedef decltype(shape) SH;
    const int64_t items = (int64_t)(max_rows / SH::TILE + 1 + (S < max_rows ? S : max_rows)) *
                          ceil_div(N, SH::TILE);
    grouped_grad_f32_kernel<false, SH><<<grid32(items), kThreads32, 0, stream>>>(p);
  };
  if (few_tiles((int64_t)(max_rows / Large32::TILE + (S < max_rows ? S : max_rows)) *
                ceil_div(N, Large32::TILE)))
    go(Small32{});
  else
    go(Large32{});
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
  p.splits = grad_splits(S, max_rows, M, N, kGradTileF32);
  p.out = p.splits > 1 ? ws : dw;
  p.out_bf16 = p.splits > 1 ? 0 : !dw_f32;
  p.accumulate = p.splits > 1 ? 0 : accumulate;
  auto go = [&](auto shape) {
    typedef decltype(shape) SH;
    const int64_t items = (int64_t)S * p.splits * ceil_div(M, SH::TILE) * ceil_div(N, SH::TILE);
    grouped_grad_f32_kernel<true, SH><<<grid32(items), kThreads32, 0, stream>>>(p);
  };
  if (few_tiles((int64_t)S * p.splits * ceil_div(M, Large32::TILE) * ceil_div(N, Large32::TILE)))
    go(Small32{});
  else
    go(Large32{});
  if (p.splits > 1)
    return launch_fold_splits(static_cast<const float*>(ws), p.splits, (size_t)S * M * N, dw, dw_f32,
                              accumulate, stream);
  return launch_status();
}

}  // namespace moe
