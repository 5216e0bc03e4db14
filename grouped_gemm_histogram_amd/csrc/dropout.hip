// dropout.hip -- dropout of a contiguous array, added to a residual:
//
//   out[i] = residual[i] + (kept(i) ? x[i] / (1 - p) : 0)
//
// The mask is recomputed from (seed, offset, i) wherever it is needed (dropout_device.h) and never
// stored, so the backward pass is the same kernel on the gradient without a residual.  A
// dropped element is selected away, not multiplied by zero: an infinity or NaN there is gone.
// A thread has eight consecutive elements, one counter block; the rest of n % 8 is taken
// element by element by the thread that has the last block.
//
// Bound by HBM and the ten rounds of the generator together (the VALU is busy 73% of the time): bf16
// 8192 x 4096 with a residual takes 34 us, 5.9 TB/s; f32 1021 x 2881 without one 7.4 us for a copy's 5.

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "dropout_device.h"
#include "launch.h"
#include "rows_device.h"

namespace moe {

// eight consecutive elements of T as f32, `left` of them present
template <typename T>
__device__ __forceinline__ void load8(const T* p, long long left, float (&v)[8]) {
  constexpr int EL = kRowEl<T>;
#pragma unroll
  for (int h = 0; h < 8 / EL; ++h) {
    float f[EL];
    chunk_to_f32<T>(load_chunk<T, false>(p + h * EL, (int)std::min<long long>(left - h * EL, EL)), f);
#pragma unroll
    for (int i = 0; i < EL; ++i) v[h * EL + i] = f[i];
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, long long left, const float (&v)[8]) {
  constexpr int EL = kRowEl<T>;
#pragma unroll
  for (int h = 0; h < 8 / EL; ++h) {
    float f[EL];
#pragma unroll
    for (int i = 0; i < EL; ++i) f[i] = v[h * EL + i];
    store_chunk<T, false>(p + h * EL, chunk_from_f32<T>(f), (int)std::min<long long>(left - h * EL, EL));
  }
}

// x, residual and out may be the same array
template <typename TX, typename TR, bool kRes, typename TO>
__global__ __launch_bounds__(256) void dropout_add_kernel(const TX* x, const TR* residual, long long n, Drop d,
                                                          const uint64_t* __restrict__ rng, TO* out) {
  const uint64_t seed = rng[0], offset = rng[1];
  const long long blocks = (n + 7) / 8;
  for (long long b = (long long)blockIdx.x * 256 + threadIdx.x; b < blocks; b += (long long)gridDim.x * 256) {
    const long long i0 = b * 8, left = n - i0;
    float v[8], r[8];
    load8<TX>(x + i0, left, v);
    if constexpr (kRes) load8<TR>(residual + i0, left, r);
    const uint32_t keep = keep_bits(offset + (uint64_t)b, seed, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float base = kRes ? r[j] : 0.0f;
      v[j] = (keep >> j & 1) ? fmaf(v[j], d.scale, base) : base;
    }
    store8<TO>(out + i0, left, v);
  }
}

Drop make_drop(double p) {
  const double t = nearbyint(p * 4294967296.0);   // round(p * 2^32), ties to even
  const unsigned long long u = (unsigned long long)t;
  return Drop{(uint32_t)(u >> 16), (uint32_t)(u & 0xffffu), p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f};
}

hipError_t launch_dropout_add(const DropoutLaunch& p, hipStream_t stream) {
  if (p.n <= 0) return hipSuccess;
  const Drop d = make_drop(p.p);
  const long long blocks = (p.n + 2047) / 2048;
  const dim3 grid((unsigned)std::min<long long>(blocks, 256 * 16)), block(256);
  auto go = [&](auto* x, auto* res, auto* out) {
    using TX = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    using TR = std::remove_const_t<std::remove_pointer_t<decltype(res)>>;
    using TO = std::remove_pointer_t<decltype(out)>;
    if (res)
      hipLaunchKernelGGL((dropout_add_kernel<TX, TR, true, TO>), grid, block, 0, stream, x, res, p.n, d, p.rng, out);
    else
      hipLaunchKernelGGL((dropout_add_kernel<TX, TX, false, TO>), grid, block, 0, stream, x, x, p.n, d, p.rng, out);
    return hipGetLastError();
  };
  auto with_out = [&](auto* x, auto* res) {
    return p.out_bf16 ? go(x, res, static_cast<uint16_t*>(p.out)) : go(x, res, static_cast<float*>(p.out));
  };
  auto with_res = [&](auto* x) {
    return p.residual_bf16 ? with_out(x, static_cast<const uint16_t*>(p.residual))
                           : with_out(x, static_cast<const float*>(p.residual));
  };
  return p.x_bf16 ? with_res(static_cast<const uint16_t*>(p.x)) : with_res(static_cast<const float*>(p.x));
}

}  // namespace moe
