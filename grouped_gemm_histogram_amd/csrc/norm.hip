// norm.hip -- layer norm of token rows, and its root-mean-square form:
//
//   y = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//
// with mean = 0 in the root-mean-square form.  A row stays in registers between its statistics
// and its output, so x is read once; the variance is taken of the differences from the mean
// (a second sum over registers), never as a difference of two large sums.  A block walks
// rows grid-wide with the parameters of its columns in registers and the next row's loads in
// flight while the current row is reduced.
//
// Bound by HBM for many rows: bf16 8192 x 7168 takes 48 to 51 us, 4.6 to 4.9 TB/s, where a copy of as many bytes
// takes 41 to 48 (with 23 VALU operations an element, the VALU is busy 87% of the time); f32 1531 x 2881
// (rows that start at any 4 bytes) 7.9 us of 7.  Few rows are a chain of a load, the sums over the waves
// and a store: one row of 2880 in 2.5 us, 1.8 us of them the launch.  Rows that need four chunks a lane
// of bf16 or seven of f32 in sixteen waves (over 24576 elements) spill registers: bf16 4096 x 28672
// takes 163 us, 2.9 TB/s.  Not kept: a block per row instead of a walk (57 to 200 us for the 58 that
// 8192 x 7168 took before the parameters came in 16-byte loads), two or four rows per barrier (no gain).

#include <algorithm>

#include "launch.h"
#include "rows_device.h"

namespace moe {

// waves of a block
template <int W>
constexpr int kNormWaves = W < 4 ? 4 : W;

// y may be x
template <typename T, bool kVec, int W, int C>
__global__ __launch_bounds__(kNormWaves<W> * 64) void norm_kernel(
    const T* x, long long T_rows, int H, const void* __restrict__ weight, const void* __restrict__ bias,
    int w_bf16, float eps, int rms, T* y, float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  constexpr int EL = kRowEl<T>;
  constexpr int kWaves = kNormWaves<W>;
  constexpr int kSlots = kWaves / W;   // rows at a time
  __shared__ float red[2 * kMaxSums * kWaves];
  const int wave = threadIdx.x >> 6;
  const int slot = wave / W;
  const int rl = (wave % W) * kWave + lane_id();   // lane within the row
  struct Row {
    uint4 x[C];
  };
  auto load_row = [&](long long t, Row& r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * W * kWave + rl) * EL;
      r.x[c] = load_chunk<T, kVec>(x + t * H + col, t < T_rows ? H - col : 0);
    }
  };
  const long long step = (long long)gridDim.x * kSlots;
  Row cur, nxt;
  load_row((long long)blockIdx.x * kSlots + slot, nxt);
  float w[C][EL], b[C][EL];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * W * kWave + rl) * EL;
    load_params<EL>(weight, w_bf16, col, H - col, 1.0f, w[c]);
    load_params<EL>(bias, w_bf16, col, H - col, 0.0f, b[c]);
  }
  const float inv_h = 1.0f / (float)H;
  int buf = 0;   // alternates over the sums
  for (long long base = (long long)blockIdx.x * kSlots; base < T_rows; base += step) {   // same count for all waves
    const long long t = base + slot;
    cur = nxt;
    if (base + step < T_rows) load_row(t + step, nxt);
    float mean = 0.0f;
    if (!rms) {
      float s[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v[EL];
        chunk_to_f32<T>(cur.x[c], v);
#pragma unroll
        for (int i = 0; i < EL; ++i) s[0] += v[i];   // entries past the row are zero
      }
      row_sums<W>(s, red, buf ^= 1, kWaves);
      mean = s[0] * inv_h;
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int left = H - (c * W * kWave + rl) * EL;
      float v[EL];
      chunk_to_f32<T>(cur.x[c], v);
#pragma unroll
      for (int i = 0; i < EL; ++i) {
        const float d = i < left ? v[i] - mean : 0.0f;
        s[0] += d;
        s[1] = fmaf(d, d, s[1]);
      }
    }
    row_sums<W>(s, red, buf ^= 1, kWaves);
    if (t >= T_rows) continue;
    // delta: what rounding left of the mean (0 up to rounding), taken out of both moments, so
    // that a row far from zero keeps its variance and its differences
    const float delta = rms ? 0.0f : s[0] * inv_h;
    const float var = s[1] * inv_h - delta * delta;
    const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);   // a NaN stays one
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * W * kWave + rl) * EL;
      float v[EL];
      chunk_to_f32<T>(cur.x[c], v);
#pragma unroll
      for (int i = 0; i < EL; ++i) v[i] = fmaf(((v[i] - mean) - delta) * rstd, w[c][i], b[c][i]);
      // rows that start inside a 16-byte unit are stored past the caches (f32 1531 x 2881: 10.8 -> 8.1 us;
      // aligned rows gain nothing: bf16 8192 x 7168 48.0 -> 49.8 us)
      store_chunk<T, kVec, !kVec>(y + t * H + col, chunk_from_f32<T>(v), H - col);
    }
    if (rl == 0) {
      if (mean_out && !rms) mean_out[t] = mean + delta;
      if (rstd_out) rstd_out[t] = rstd;
    }
  }
}

// Fewer rows than this take one chunk a lane (up to sixteen waves a row), for the latency: 64 rows of
// bf16 2880 take 3.0 us for 3.3, 256 take 3.2 for 3.4.  From here on two chunks a lane are faster:
// 512 rows of 7168 take 5.6 us for 6.3, 4096 of 2880 13.7 for 15.6.
constexpr int kFewRows = 512;

template <typename T, bool kVec>
struct NormLauncher {
  const NormLaunch& p;
  hipStream_t stream;
  template <int W, int C>
  hipError_t operator()() const {
    constexpr int kWaves = kNormWaves<W>;
    constexpr int kSlots = kWaves / W;
    const long long blocks = (p.T + kSlots - 1) / kSlots;
    // 16 waves a CU: 8, 24 and 40 took 71, 64 and 69 us where 16 took 58 (8192 x 7168, as above)
    const unsigned grid = (unsigned)std::min<long long>(blocks, 256 * 16 / kWaves);
    hipLaunchKernelGGL((norm_kernel<T, kVec, W, C>), dim3(grid), dim3(kWaves * kWave), 0, stream,
                       static_cast<const T*>(p.x), p.T, p.H, p.weight, p.bias, p.w_bf16, p.eps, p.rms,
                       static_cast<T*>(p.y), p.mean, p.rstd);
    return hipGetLastError();
  }
};

template <typename T, bool kVec>
static hipError_t launch_norm_v(const NormLaunch& p, hipStream_t stream) {
  const int units = (p.H + kRowEl<T> - 1) / kRowEl<T>;
  const NormLauncher<T, kVec> go{p, stream};
  return p.T < kFewRows ? dispatch_row<1, kWideChunks<T>>(units, go)
                        : dispatch_row<16 / kRowEl<T>, kWideChunks<T>>(units, go);
}

template <typename T>
static hipError_t launch_norm_t(const NormLaunch& p, hipStream_t stream) {
  return p.H % kRowEl<T> == 0 ? launch_norm_v<T, true>(p, stream) : launch_norm_v<T, false>(p, stream);
}

hipError_t launch_norm(const NormLaunch& p, hipStream_t stream) {
  if (p.T <= 0) return hipSuccess;
  return p.x_bf16 ? launch_norm_t<uint16_t>(p, stream) : launch_norm_t<float>(p, stream);
}

}  // namespace moe
