// eightbit.hip -- rows to 8-bit integers with a scale each: token rows in front of the 8-bit grouped
// product (gemm.hip), and weight rows, whose scale is then the output channel's.
//
//     scale = amax * (1 / 127),   code = round(x * (127 * (1 / amax))), ties to even, each operation in f32
//
// A row stays in the registers of 1 to 16 waves between its largest value and its codes, so x is read
// once: 3 bytes an element of bf16.  The maximum is taken on the values' bits without their
// sign, which order as integers do, with NaN above infinity: a row that holds one gets a NaN or infinite
// scale and no other row notices.

#include <algorithm>

#include "launch.h"
#include "rows_device.h"

namespace moe {

namespace {

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto rotated = [](uint32_t x, auto by) {   // row_ror:by
    return (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0x120 + decltype(by)::value, 0xf, 0xf, false);
  };
  v = max(v, rotated(v, std::integral_constant<int, 8>{}));
  v = max(v, rotated(v, std::integral_constant<int, 4>{}));
  v = max(v, rotated(v, std::integral_constant<int, 2>{}));
  v = max(v, rotated(v, std::integral_constant<int, 1>{}));
  auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max((uint32_t)s[0], (uint32_t)s[1]);
  s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)s[0], (uint32_t)s[1]);
}

// four codes of x * inv: adding 1.5 * 2^23 rounds to an integer, whose low byte is the sum's
__device__ __forceinline__ uint32_t pack_codes(const float* x, float inv) {
#pragma clang fp contract(off)
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(x[i] * inv + 12582912.0f);
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);   // bytes: b0[0], b1[0], 0, 0
  return __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu) | lo;
}

template <int W>
constexpr int kQuantWaves = W < 4 ? 4 : W;

template <typename T, int W, int C>
__global__ __launch_bounds__(kQuantWaves<W> * 64) void quantize_rows_kernel(const T* __restrict__ x, long long rows,
                                                                            const int* __restrict__ valid, int H,
                                                                            uint8_t* __restrict__ codes,
                                                                            float* __restrict__ scales) {
  constexpr int EL = kRowEl<T>;
  constexpr int kWaves = kQuantWaves<W>;
  constexpr int kSlots = kWaves / W;
  __shared__ uint32_t red[kWaves];
  const int wave = threadIdx.x >> 6;
  const long long t = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * kSlots + wave / W;
  const int rl = (wave % W) * kWave + lane_id();
  const long long last = valid ? min(rows, (long long)max(*valid, 0)) : rows;
  const bool live = t < last;
  uint4 raw[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * W * kWave + rl) * EL;
    raw[c] = load_chunk<T, true>(x + t * H + col, live ? H - col : 0);
  }
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float v[EL];
    chunk_to_f32<T>(raw[c], v);
#pragma unroll
    for (int i = 0; i < EL; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  }
  top = wave_max(top);
  if constexpr (W > 1) {
    if (lane_id() == 0) red[wave] = top;
    __syncthreads();
    top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) top = max(top, red[(wave / W) * W + i]);
  }
  if (!live) return;
  const float amax = __uint_as_float(top);
  const bool none = amax < 0x1p-100f;   // a row of zeros: 1 / amax is finite for all others
  const float scale = none ? 1.0f : amax * (1.0f / 127.0f);
  const float inv = none ? 0.0f : 127.0f * (1.0f / amax);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * W * kWave + rl) * EL;
    if (col >= H) continue;
    float v[EL];
    chunk_to_f32<T>(raw[c], v);
    uint32_t w[EL / 4];
#pragma unroll
    for (int i = 0; i < EL / 4; ++i) w[i] = pack_codes(v + 4 * i, inv);
    __builtin_memcpy(codes + t * H + col, w, EL);
  }
  if (rl == 0) scales[t] = scale;
}

template <typename T>
struct QuantLauncher {
  const QuantizeLaunch& p;
  hipStream_t stream;
  template <int W, int C>
  hipError_t operator()() const {
    constexpr int kSlots = kQuantWaves<W> / W;
    constexpr long long kMaxX = 1 << 20;   // a grid's axis has fewer than 2^32 threads
    const long long blocks = (p.rows + kSlots - 1) / kSlots;
    hipLaunchKernelGGL((quantize_rows_kernel<T, W, C>),
                       dim3((unsigned)std::min(blocks, kMaxX), (unsigned)((blocks + kMaxX - 1) / kMaxX)),
                       dim3(kQuantWaves<W> * kWave), 0, stream, static_cast<const T*>(p.x), p.rows, p.valid, p.H,
                       static_cast<uint8_t*>(p.codes), p.scales);
    return hipGetLastError();
  }
};

// few rows spread over more waves, one chunk a lane (as the layer norm's rows do)
constexpr int kFewRows = 512;

template <typename T>
hipError_t launch_quantize_t(const QuantizeLaunch& p, hipStream_t stream) {
  const int units = p.H / kRowEl<T>;
  const QuantLauncher<T> go{p, stream};
  return p.rows < kFewRows ? dispatch_row<1, kWideChunks<T>>(units, go)
                           : dispatch_row<16 / kRowEl<T>, kWideChunks<T>>(units, go);
}

}  // namespace

hipError_t launch_quantize_eightbit(const QuantizeLaunch& p, hipStream_t stream) {
  if (p.rows <= 0) return hipSuccess;
  return p.x_bf16 ? launch_quantize_t<uint16_t>(p, stream) : launch_quantize_t<float>(p, stream);
}

}  // namespace moe
