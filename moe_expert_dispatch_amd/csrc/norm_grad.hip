// Gradient of the root-mean-square norm and of the layer norm.
//
//   n = (x - m) r   (RMS: m = 0), r = 1 / sqrt(mean (x - m)^2 + eps)
//   g = dy * gamma
//   dx = r (g - mean g - n mean(g n)) + dresidual   (RMS: without mean g)
//   dgamma = sum over rows of dy * n,  dbeta = sum over rows of dy
//
// The row's mean and deviation are formed again from x, which is read anyway,
// so nothing has to be kept from the forward pass. A block goes from row to
// row with its columns' sums for dgamma and dbeta in registers; each block
// writes one row of partial sums, and a second kernel adds those in order.
// Every sum's order depends on T and H alone.
//
// Bound by the bytes, two or three rows read and one written: 16384 rows of 4096
// bf16 with dresidual 124 to 128 us (4.2 to 4.3 TB/s; the sums of the row before
// and the loads of the next one overlap only as far as the registers of two blocks
// of eight waves a compute unit reach), 8192 rows of 5120 RMS, dresidual too, 67 (5.0),
// 777 rows of 2056 f32 without it 11.2; the second kernel 4 to 5 us.
#include <algorithm>

#include "norm_row.h"

namespace moe {
namespace {

template <typename XT, bool CENTRED, int VPT, int L>
__global__ __launch_bounds__(L == 0 ? 1024 : kNormGroupThreads) void norm_backward_kernel(
    const XT* dy, const XT* x, const XT* __restrict__ gamma, const XT* dresidual, int T, int H,
    float eps, XT* dx, float* __restrict__ pg, float* __restrict__ pb, int part_stride) {
  __shared__ RowParts part;
  constexpr int kRows = L == 0 ? 1 : kNormGroupThreads / (L == 0 ? 1 : L);
  const int group = L == 0 ? 0 : threadIdx.x / (L == 0 ? 1 : L);
  const int first = L == 0 ? threadIdx.x : threadIdx.x % (L == 0 ? 1 : L);
  const int stride = L == 0 ? blockDim.x : L;
  const int nvec = H / 8;
  const float over = 1.0f / (float)H;
  const int64_t step = (int64_t)gridDim.x * kRows;
  float ag[VPT][8] = {}, ab[VPT][8] = {};
  // A row's vectors are asked for while the row before is worked on (rows of one
  // vector a thread: for wider ones the registers would not hold them).
  constexpr bool kAhead = VPT == 1;
  typedef decltype(raw8(x)) Raw;
  Raw nx = {}, nd = {}, nr = {}, ng = {};
  constexpr bool kGuess = CENTRED && L == 0 && VPT == 1;
  const bool mine = first < nvec;
  const bool add = dresidual != nullptr && dx != nullptr;
  auto ask = [&](int64_t t) {
    if (t < T && mine) {
      const size_t at = (size_t)t * H + first * 8;
      nx = raw8(x + at);
      if constexpr (kGuess) ng = raw8(x + (size_t)t * H);
      nd = raw8(dy + at);
      if (add) nr = raw8(dresidual + at);
    }
  };
  int64_t t = (int64_t)blockIdx.x * kRows + group;
  if constexpr (kAhead) ask(t);
  for (; t < T; t += step) {
    const size_t row = (size_t)t * H;
    float h[VPT][8] = {}, d[VPT][8] = {};
    Raw res = nr;
    float guess = 0.f;
    if constexpr (kGuess) {
      float v[8];
      unpack8(ng, v);
      guess = mean8(v);
    }
    if constexpr (kAhead) {
      if (mine) {
        unpack8(nx, h[0]);
        unpack8(nd, d[0]);
      }
      ask(t + step);
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = first + j * stride;
        if (v < nvec) {
          load8(x + row + v * 8, h[j]);
          load8(dy + row + v * 8, d[j]);
        }
      }
    }
    const float r = normalize_row<CENTRED, VPT, L>(h, first, stride, nvec, H, eps, part, guess);
    float sg = 0.f, sn = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = first + j * stride;
      if (v < nvec) {
        float w[8];
        load8(gamma + v * 8, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ag[j][i] = fmaf(d[j][i], h[j][i], ag[j][i]);
          if constexpr (CENTRED) ab[j][i] += d[j][i];
          d[j][i] *= w[i];
          sn = fmaf(d[j][i], h[j][i], sn);
          if constexpr (CENTRED) sg += d[j][i];
        }
      }
    }
    const float2 sums = lanes_sum2<L>(sn, sg, part.grad);
    sn = sums.x * over;
    sg = sums.y * over;
    if (dx != nullptr) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = first + j * stride;
        if (v < nvec) {
          float o[8] = {};
          if (dresidual != nullptr) {
            if constexpr (kAhead) unpack8(res, o);
            else load8(dresidual + row + v * 8, o);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float c = CENTRED ? fmaf(-h[j][i], sn, d[j][i] - sg) : fmaf(-h[j][i], sn, d[j][i]);
            o[i] = fmaf(c, r, o[i]);
          }
          store8(dx + row + v * 8, o);
        }
      }
    }
  }
  if (pg == nullptr && pb == nullptr) return;
  const size_t at = (size_t)blockIdx.x * part_stride;
  if constexpr (L == 0) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = first + j * stride;
      if (v < nvec) {
        if (pg != nullptr) store8(pg + at + v * 8, ag[j]);
        if (CENTRED && pb != nullptr) store8(pb + at + v * 8, ab[j]);
      }
    }
  } else {  // the block's groups in order
    constexpr int W = L * 8;
    __shared__ float both[2][kRows][W];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      both[0][group][first * 8 + i] = ag[0][i];
      both[1][group][first * 8 + i] = ab[0][i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < H; c += kNormGroupThreads) {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        a += both[0][k][c];
        b += both[1][k][c];
      }
      if (pg != nullptr) pg[at + c] = a;
      if (CENTRED && pb != nullptr) pb[at + c] = b;
    }
  }
}

// The whole gradient of a few rows in one launch: blocks 0 .. T-1 give a row of
// dx each, the others 64 columns of dgamma and dbeta each, for which they form
// every row's mean and deviation once more, a wave to a row: time that grows with
// the rows and their width (take_few).
constexpr int kFewRows = 16;
constexpr int kColumns = 64;  // of a block

// The first vectors of a wave's row, and the row's first 8 values for all lanes.
template <typename XT>
struct WaveRow {
  decltype(raw8((const XT*)nullptr)) q[4], f;
  __device__ __forceinline__ void ask(const XT* x, int nvec) {
    f = raw8(x);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (lane_id() + u * kWave < nvec) q[u] = raw8(x + (lane_id() + u * kWave) * 8);
  }
};

// A wave's row: its mean and 1 / deviation, in f64 from f32 sums or, where those
// will not do (normalize_row), from f64 ones.
template <typename XT, bool CENTRED>
__device__ __forceinline__ void wave_row(const XT* x, WaveRow<XT> w, int nvec, int H, float eps,
                                         double* mean, double* r) {
  const float width = (float)H;
  float m = 0.f, d = 0.f, ss = 0.f, var = 0.f;
  auto spread = [&]() {  // w holds the first vectors
    float sd = 0.f;
    ss = 0.f;
    for (int v0 = lane_id(); v0 < nvec; v0 += 4 * kWave) {  // four vectors in flight
      if (v0 >= 4 * kWave) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (v0 + u * kWave < nvec) w.q[u] = raw8(x + (v0 + u * kWave) * 8);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (v0 + u * kWave >= nvec) continue;
        float h[8];
        unpack8(w.q[u], h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float c = CENTRED ? h[i] - m : h[i];
          ss = fmaf(c, c, ss);
          sd += c;
        }
      }
    }
    ss = wave_sum(ss);
    if constexpr (CENTRED) d = wave_sum(sd) / width;
    var = (CENTRED ? fmaxf(ss / width - d * d, 0.f) : ss / width) + eps;
  };
  if constexpr (CENTRED) {
    float h[8];
    unpack8(w.f, h);
    m = mean8(h);
  }
  spread();
  if constexpr (CENTRED) {
    if (!(var - eps >= d * d)) {
      m += d;
      if (nvec > 4 * kWave) w.ask(x, nvec);
      spread();
    }
  }
  if (var >= kLeastSquares && var >= d * d && ss < INFINITY) {
    *mean = (double)m + (double)d;
    *r = (double)(1.0f / sqrtf(var));  // in f64 it took a wave 1 us a row
    return;
  }
  double at = 0.0;
  if constexpr (CENTRED) {
    for (int v = lane_id(); v < nvec; v += kWave) {
      float h[8];
      load8(x + v * 8, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) at += (double)h[i];
    }
    at = lanes_sum_f64<64>(at, nullptr) / H;
  }
  double sq = 0.0;
  for (int v = lane_id(); v < nvec; v += kWave) {
    float h[8];
    load8(x + v * 8, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double c = (double)h[i] - at;
      sq = fma(c, c, sq);
    }
  }
  *mean = at;
  *r = 1.0 / sqrt(lanes_sum_f64<64>(sq, nullptr) / H + (double)eps);
}

template <typename XT, bool CENTRED>
__global__ __launch_bounds__(1024) void norm_backward_few_kernel(
    const XT* dy, const XT* x, const XT* __restrict__ gamma, const XT* dresidual, int T, int H,
    float eps, int row_blocks, XT* dx, float* __restrict__ dgamma, float* __restrict__ dbeta) {
  const int nvec = H / 8;
  if ((int)blockIdx.x < row_blocks) {
    __shared__ RowParts part;
    const size_t at = (size_t)blockIdx.x * H + threadIdx.x * 8;
    const bool mine = (int)threadIdx.x < nvec;
    float h[1][8] = {}, d[8] = {}, o[8] = {}, w[8] = {}, guess = 0.f;
    if constexpr (CENTRED) {
      float v[8];
      load8(x + (size_t)blockIdx.x * H, v);
      guess = mean8(v);
    }
    if (mine) {
      load8(x + at, h[0]);
      load8(dy + at, d);
      if (dresidual != nullptr) load8(dresidual + at, o);
      load8(gamma + threadIdx.x * 8, w);
    }
    const float r =
        normalize_row<CENTRED, 1, 0>(h, threadIdx.x, blockDim.x, nvec, H, eps, part, guess);
    float sg = 0.f, sn = 0.f;
    if (mine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] *= w[i];
        sn = fmaf(d[i], h[0][i], sn);
        sg += d[i];
      }
    }
    const float2 sums = lanes_sum2<0>(sn, sg, part.grad);
    sn = sums.x / (float)H;
    sg = CENTRED ? sums.y / (float)H : 0.f;
    if (mine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(fmaf(-h[0][i], sn, d[i] - sg), r, o[i]);
      store8(dx + at, o);
    }
    return;
  }
  __shared__ double mean[kFewRows], dev[kFewRows];
  __shared__ float sums[2][16][kColumns];
  const int wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
  if (wave < T) {  // the block has a wave for each row
    const XT* row = x + (size_t)wave * H;
    WaveRow<XT> w;
    w.ask(row, nvec);
    double m, r;
    wave_row<XT, CENTRED>(row, w, nvec, H, eps, &m, &r);
    if (lane_id() == 0) {
      mean[wave] = m;
      dev[wave] = r;
    }
  }
  __syncthreads();
  // 8 lanes to the 64 columns of a row, every 8th row of the wave's
  const int v = (blockIdx.x - row_blocks) * (kColumns / 8) + (lane_id() & 7);
  float ag[8] = {}, ab[8] = {};
  if (v < nvec) {
    for (int t = threadIdx.x / 8; t < T; t += blockDim.x / 8) {
      float h[8], d[8];
      load8(x + (size_t)t * H + v * 8, h);
      load8(dy + (size_t)t * H + v * 8, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = (float)((CENTRED ? (double)h[i] - mean[t] : (double)h[i]) * dev[t]);
        ag[i] = fmaf(d[i], n, ag[i]);
        ab[i] += d[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = 8; o < kWave; o *= 2) {
      ag[i] += __shfl_xor(ag[i], o, kWave);
      if constexpr (CENTRED) ab[i] += __shfl_xor(ab[i], o, kWave);
    }
    if (lane_id() < 8) {
      sums[0][wave][lane_id() * 8 + i] = ag[i];
      sums[1][wave][lane_id() * 8 + i] = ab[i];
    }
  }
  __syncthreads();
  const int c = (blockIdx.x - row_blocks) * kColumns + (threadIdx.x & 63);
  const int which = threadIdx.x / kColumns;
  if (which > 1 || c >= H) return;
  float* out = which == 0 ? dgamma : dbeta;
  if (out == nullptr) return;
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += sums[which][w][threadIdx.x & 63];
  out[c] = s;
}

// out[c] = the sum over n rows of part [n, H], or zero for none: 32 lines of a
// block add every 32nd row of 32 columns, 16 rows asked for at a time, then the
// lines are added in order.
__global__ __launch_bounds__(256) void fold_columns_kernel(const float* __restrict__ pg,
                                                           const float* __restrict__ pb, int n,
                                                           int H, float* __restrict__ dgamma,
                                                           float* __restrict__ dbeta) {
  constexpr int kLines = 32, kAhead = 16;
  const float* part = blockIdx.y == 0 ? pg : pb;
  float* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (out == nullptr) return;
  __shared__ float4 lines[kLines][8];
  const int line = threadIdx.x / 8, at = threadIdx.x % 8;
  const int c = (blockIdx.x * 8 + at) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < H) {
    for (int k0 = line; k0 < n; k0 += kLines * kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * kLines;
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < n) v[u] = *reinterpret_cast<const float4*>(part + (size_t)k * H + c);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        s.x += v[u].x;
        s.y += v[u].y;
        s.z += v[u].z;
        s.w += v[u].w;
      }
    }
  }
  lines[line][at] = s;
  __syncthreads();
  if (line != 0 || c >= H) return;
#pragma unroll
  for (int k = 1; k < kLines; ++k) {
    const float4 v = lines[k][at];
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  *reinterpret_cast<float4*>(out + c) = s;
}

// Blocks that share the rows: whole rounds of 256 compute units with about 16
// waves each (8192 rows of 5120, ten waves a row: 512 blocks 96 us, 409 117), and
// 16 rows a block, or no more than 8 MB of partial sums, which are written and
// read once more (2048 rows of 2048: 512 blocks 20 us, 1024 23).
int norm_blocks(int T, int H) {
  if (T == 0) return 0;
  const int L = norm_lanes(H / 8);
  const int waves = L == 0 ? std::min(16, ceil_div(H / 8, kWave)) : kNormGroupThreads / kWave;
  const int64_t rows = L == 0 ? 1 : kNormGroupThreads / L;
  const int64_t most = std::min(256 * std::clamp((16 + waves / 2) / waves, 1, 4),
                                std::max({256, (1 << 20) / H, T / 16}));
  // as many rows a block as it takes, evenly: no more partial sums than that
  const int64_t sets = (T + rows - 1) / rows, each = (sets + most - 1) / most;
  return (int)((sets + each - 1) / each);
}

// Up to there one launch takes the GPU no longer than two, whose second one also
// costs the host 4 us a call (11 and 15 us issued one after the other, 10 and 14 RMS).
// One launch and two, us on the GPU, layer norm bf16: 12 rows of 512 to 2048 4.7 to
// 5.2 and 6.0 to 6.2, of 8192 7.8 and 8.3; 16 rows of 512 5.4 and 6.1, of 2048 6.1 and
// 6.2, of 4096 6.8 and 6.7, of 8192 8.4 and 8.5 (f32 9.7 and 9.1); above, with several
// rows a wave, 24 of 512 6.3 and 5.9, of 2048 7.0 and 6.2, of 8192 10.1 and 8.8, 64 of
// 2048 11.7 and 6.5. RMS 16 rows of 512 to 8192 4.1 to 6.1 and 5.6 to 6.8, 24 of 2048
// 5.1 and 5.6, 64 8.1 and 5.7. Rows that one block of the other form holds need no
// second launch there: 16 of 128 2.8 us (here 5.7), 4 of 512 3.1 (3.9).
bool take_few(int T, int H) {
  return T <= kFewRows && H <= 8192 && norm_blocks(T, H) > 1;
}

template <typename XT, bool CENTRED>
void launch_few(const void* dy, const void* x, const void* gamma, const void* dresidual, int T,
                int H, float eps, void* dx, float* dgamma, float* dbeta, hipStream_t stream) {
  // vectors of a row for its block, and a wave a row for the columns' blocks
  const int threads = std::max({256, ceil_div(H / 8, kWave) * kWave, T * kWave});
  const int columns = dgamma != nullptr || dbeta != nullptr ? ceil_div(H, kColumns) : 0;
  auto go = [&](int rows, int cols) {
    if (rows + cols > 0)
      norm_backward_few_kernel<XT, CENTRED><<<rows + cols, threads, 0, stream>>>(
          static_cast<const XT*>(dy), static_cast<const XT*>(x), static_cast<const XT*>(gamma),
          static_cast<const XT*>(dresidual), T, H, eps, rows, static_cast<XT*>(dx), dgamma, dbeta);
  };
  const int rows = dx != nullptr ? T : 0;
  if (dx != x && dx != dy) {
    go(rows, columns);
  } else {  // the columns' blocks read what the rows' overwrite
    go(0, columns);
    go(rows, 0);
  }
}

template <typename XT, bool CENTRED>
void launch_typed(const void* dy, const void* x, const void* gamma, const void* dresidual, int T,
                  int H, float eps, void* dx, float* pg, float* pb, int part_stride, int blocks,
                  hipStream_t stream) {
  const int nvec = H / 8;
  auto go = [&](auto vpt, auto lanes) {
    constexpr int VPT = decltype(vpt)::value, L = decltype(lanes)::value;
    const int threads = L == 0 ? ceil_div(ceil_div(nvec, VPT), kWave) * kWave : kNormGroupThreads;
    norm_backward_kernel<XT, CENTRED, VPT, L><<<blocks, threads, 0, stream>>>(
        static_cast<const XT*>(dy), static_cast<const XT*>(x), static_cast<const XT*>(gamma),
        static_cast<const XT*>(dresidual), T, H, eps, static_cast<XT*>(dx), pg, pb, part_stride);
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

size_t norm_backward_workspace_bytes(int T, int H) {
  if (take_few(T, H)) return 0;
  const int blocks = norm_blocks(T, H);
  return blocks > 1 ? (size_t)blocks * H * 2 * sizeof(float) : 0;
}

moe_status_t launch_norm_backward(bool centred, const void* dy, const void* x, const void* gamma,
                                  const void* dresidual, bool bf16, int T, int H, float eps,
                                  void* dx, float* dgamma, float* dbeta, void* ws,
                                  hipStream_t stream) {
  const bool sums = dgamma != nullptr || dbeta != nullptr;
  if (T == 0 && !sums) return MOE_OK;
  const bool few = take_few(T, H);
  const int blocks = norm_blocks(T, H);
  float* pg = blocks == 1 ? dgamma : static_cast<float*>(ws);
  float* pb = blocks == 1 ? dbeta : static_cast<float*>(ws) + (size_t)blocks * H;  // of no rows: unread
  if (T > 0) {
    float* kg = dgamma != nullptr ? pg : nullptr;
    float* kb = dbeta != nullptr ? pb : nullptr;
    auto go = [&](auto kind, auto c) {
      typedef typename decltype(kind)::type XT;
      if (few)
        launch_few<XT, decltype(c)::value>(dy, x, gamma, dresidual, T, H, eps, dx, dgamma, dbeta,
                                           stream);
      else
        launch_typed<XT, decltype(c)::value>(dy, x, gamma, dresidual, T, H, eps, dx, kg, kb, H,
                                             blocks, stream);
    };
    struct B16 { typedef uint16_t type; };
    struct F32 { typedef float type; };
    if (bf16 && centred) go(B16{}, std::true_type{});
    else if (bf16) go(B16{}, std::false_type{});
    else if (centred) go(F32{}, std::true_type{});
    else go(F32{}, std::false_type{});
  }
  if (sums && blocks != 1 && !few)
    fold_columns_kernel<<<dim3(ceil_div(H, 32), dbeta != nullptr ? 2 : 1), 256, 0, stream>>>(
        pg, pb, blocks, H, dgamma, dbeta);
  return launch_status();
}

}  // namespace moe
