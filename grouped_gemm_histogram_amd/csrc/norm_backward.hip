// norm_backward.hip -- gradients of the layer norm in norm.hip.  With xhat = (x - mean) * rstd
// and g = weight * dy,
//
//   dx      = rstd * (g - mean(g) - xhat * mean(g * xhat))    (no mean(g) in the rms form)
//   dweight = sum over rows of dy * xhat,   dbias = sum over rows of dy
//
// One pass: a block walks rows grid-wide with x and dy read once into registers (the next row's
// loads in flight meanwhile), writes dx, and adds each row to f32 sums of its columns that stay in
// registers until the block's last row.  The sums go to the workspace, one row per row slot, and
// a second kernel adds those rows in a fixed order: no atomics, so results do not vary.
//
// Bound by HBM: x and dy read, dx written.  bf16 8192 x 7168 takes 68 us (5.2 TB/s) and 5.0 for the
// sums of the partial rows; 4096 x 2880 17 and 4.0 (f32 26 and 4.0), where its 71 MB alone would take 12
// to 14: with 16 rows a block, filling and draining the pipeline and the columns' sums show.  One row of
// 2880 takes 5.1 and 2.3.  The columns' sums of both gradients are made also where only one is asked for.
// Two, three and four rows' loads in flight ahead of the current row's sums are slower than one (by 0.9, 1.9
// and 2.9 us).  The columns' sums stored word by word cost 2 to 3 us more.

#include <algorithm>

#include "launch.h"
#include "rows_device.h"

namespace moe {

// waves of a block: with 16 in every block the columns' sums spill (126 us for 71 at 8192 x 7168)
template <int W>
constexpr int kNbWaves = W < 8 ? 8 : W;

// dx may be dy or x
template <typename T, bool kVec, int W, int C>
__global__ __launch_bounds__(kNbWaves<W> * 64) void norm_backward_kernel(
    const T* dy, const T* x, long long T_rows, int H, const void* __restrict__ weight,
    int w_bf16, const float* __restrict__ mean_in, const float* __restrict__ rstd_in, int rms, T* dx,
    float* __restrict__ part) {
  constexpr int EL = kRowEl<T>;
  constexpr int kWaves = kNbWaves<W>;
  constexpr int kSlots = kWaves / W;
  __shared__ float red[2 * kMaxSums * kWaves];
  __shared__ float merge[kSlots > 1 ? kSlots / 2 * W * kWave : 1][kSlots > 1 ? C * EL + 1 : 1];   // a row a thread, odd
  const int wave = threadIdx.x >> 6;
  const int slot = wave / W;
  const int rl = (wave % W) * kWave + lane_id();   // lane within the row
  float w[C][EL], dw[C][EL], db[C][EL];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * W * kWave + rl) * EL;
    load_params<EL>(weight, w_bf16, col, H - col, 1.0f, w[c]);
#pragma unroll
    for (int i = 0; i < EL; ++i) dw[c][i] = db[c][i] = 0.0f;
  }
  const float inv_h = 1.0f / (float)H;
  struct Row {
    uint4 x[C], dy[C];
    float mean, rstd;
  };
  auto load_row = [&](long long t, Row& r) {
    const bool in = t < T_rows;
    r.mean = in && !rms ? mean_in[t] : 0.0f;
    r.rstd = in ? rstd_in[t] : 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * W * kWave + rl) * EL;
      r.x[c] = load_chunk<T, kVec>(x + t * H + col, in ? H - col : 0);
      r.dy[c] = load_chunk<T, kVec>(dy + t * H + col, in ? H - col : 0);
    }
  };
  const long long step = (long long)gridDim.x * kSlots;
  int buf = 0;   // alternates over the sums
  Row cur, nxt;
  load_row((long long)blockIdx.x * kSlots + slot, nxt);
  for (long long base = (long long)blockIdx.x * kSlots; base < T_rows; base += step) {   // same count for all waves
    const long long t = base + slot;
    cur = nxt;
    if (base + step < T_rows) load_row(t + step, nxt);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float xv[EL], gv[EL];
      chunk_to_f32<T>(cur.x[c], xv);
      chunk_to_f32<T>(cur.dy[c], gv);
#pragma unroll
      for (int i = 0; i < EL; ++i) {   // entries past the row have dy = 0
        const float xhat = (xv[i] - cur.mean) * cur.rstd;
        dw[c][i] = fmaf(gv[i], xhat, dw[c][i]);
        db[c][i] += gv[i];
        const float g = gv[i] * w[c][i];
        s1 += g;
        s2 = fmaf(g, xhat, s2);
      }
    }
    float s[2] = {s1, s2};
    row_sums<W>(s, red, buf ^= 1, kWaves);
    const float m1 = rms ? 0.0f : s[0] * inv_h, m2 = s[1] * inv_h;
    if (t < T_rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * W * kWave + rl) * EL;
        float xv[EL], gv[EL];
        chunk_to_f32<T>(cur.x[c], xv);
        chunk_to_f32<T>(cur.dy[c], gv);
#pragma unroll
        for (int i = 0; i < EL; ++i) {
          const float xhat = (xv[i] - cur.mean) * cur.rstd;
          gv[i] = cur.rstd * (fmaf(-xhat, m2, gv[i] * w[c][i]) - m1);
        }
        store_chunk<T, kVec>(dx + t * H + col, chunk_from_f32<T>(gv), H - col);
      }
    }
  }
  if (!part) return;
  // the slots' sums in a tree: the upper half of the slots left hands its sums to the lower
  const int at = (slot * W + wave % W) * kWave + lane_id();   // thread of the block, by slot
#pragma unroll
  for (int half = kSlots / 2; half >= 1; half /= 2) {
    auto exchange = [&](float (&v)[C][EL]) {
      __syncthreads();
      if (slot >= half && slot < 2 * half)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < EL; ++i) merge[at - half * W * kWave][c * EL + i] = v[c][i];
      __syncthreads();
      if (slot < half)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < EL; ++i) v[c][i] += merge[at][c * EL + i];
    };
    exchange(dw);
    exchange(db);
  }
  if (slot == 0) {
    float* pw = part + (long long)blockIdx.x * 2 * H;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * W * kWave + rl) * EL;
      if (col + EL <= H) {   // in 16-byte stores
        __builtin_memcpy(pw + col, dw[c], sizeof(dw[c]));
        __builtin_memcpy(pw + H + col, db[c], sizeof(db[c]));
      } else {
#pragma unroll
        for (int i = 0; i < EL; ++i)
          if (col + i < H) {
            pw[col + i] = dw[c][i];
            pw[H + col + i] = db[c][i];
          }
      }
    }
  }
}

// dweight[h] and dbias[h] = the sums over the P partial rows [P][2H], each wave every 16th row,
// the waves' sums in wave order.  A block has 64 columns; 32 columns and 32 groups of rows take as
// long (4.0 us at 4096 x 2880, 4.7 at 8192 x 7168), 16 columns 4.0 and 6.2.
__global__ __launch_bounds__(1024) void norm_grad_sum_kernel(const float* __restrict__ part, int P, int H,
                                                             void* __restrict__ dweight, void* __restrict__ dbias,
                                                             int out_bf16) {
  __shared__ float sums[16][kWave];
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const int col = blockIdx.x * kWave + lane;
  float s = 0.0f;
  if (col < 2 * H) {
#pragma unroll 8
    for (int p = wave; p < P; p += 16) s += part[(size_t)p * 2 * H + col];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < 2 * H) {
    s = sums[0][lane];
#pragma unroll
    for (int i = 1; i < 16; ++i) s += sums[i][lane];
    void* out = col < H ? dweight : dbias;
    const int h = col < H ? col : col - H;
    if (out) {
      if (out_bf16)
        static_cast<uint16_t*>(out)[h] = f32_to_bf16_bits(s);
      else
        static_cast<float*>(out)[h] = s;
    }
  }
}

// blocks of a launch, each with one row of partial sums; 512 take 81 us for 71 at 8192 x 7168 and 24.6
// for 20.2 at 4096 x 2880
constexpr int kPartRows = 256;

template <typename T, bool kVec>
struct NormBackwardLauncher {
  const NormBackwardLaunch& p;
  hipStream_t stream;
  template <int W, int C>
  hipError_t operator()() const {
    constexpr int kSlots = kNbWaves<W> / W;
    const unsigned grid = (unsigned)std::min<long long>((p.T + kSlots - 1) / kSlots, kPartRows);
    const bool sums = p.dweight || p.dbias;
    if (p.T > 0)
      hipLaunchKernelGGL((norm_backward_kernel<T, kVec, W, C>), dim3(grid), dim3(kNbWaves<W> * kWave), 0, stream,
                         static_cast<const T*>(p.dy), static_cast<const T*>(p.x), p.T, p.H, p.weight, p.w_bf16,
                         p.mean, p.rstd, p.rms, static_cast<T*>(p.dx), sums ? p.part : nullptr);
    if (sums)
      hipLaunchKernelGGL(norm_grad_sum_kernel, dim3((2 * p.H + kWave - 1) / kWave), dim3(1024), 0, stream, p.part,
                         (int)grid, p.H, p.dweight, p.dbias, p.grad_bf16);
    return hipGetLastError();
  }
};

template <typename T>
static hipError_t launch_norm_backward_t(const NormBackwardLaunch& p, hipStream_t stream) {
  const int units = (p.H + kRowEl<T> - 1) / kRowEl<T>;
  // chunks a lane before a row takes more waves.  Three of bf16: two spill from 8192 elements on, where
  // 16 waves leave 128 registers (4096 x 8200 takes 80 us for 39, x 12288 119 for 59; narrower rows
  // are equal).  Wider rows do spill: x 16384 145 us, x 20480 470, f32 2048 x 16384 140.
  constexpr int kMaxC = sizeof(T) == 2 ? 3 : 4;
  if (p.H % kRowEl<T> == 0) return dispatch_row<kMaxC, kWideChunks<T>>(units, NormBackwardLauncher<T, true>{p, stream});
  return dispatch_row<kMaxC, kWideChunks<T>>(units, NormBackwardLauncher<T, false>{p, stream});
}

hipError_t launch_norm_backward(const NormBackwardLaunch& p, hipStream_t stream) {
  return p.x_bf16 ? launch_norm_backward_t<uint16_t>(p, stream) : launch_norm_backward_t<float>(p, stream);
}

size_t norm_backward_workspace_bytes(long long T, int H) {
  return (size_t)std::min<long long>(T, kPartRows) * 2 * H * sizeof(float);
}

}  // namespace moe
