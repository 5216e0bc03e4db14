// rows_device.h -- reading and writing token rows 16 bytes a lane, and sums over the waves of a row.
//
// A row of H elements is held by W waves with C chunks a lane: chunk c of row lane r covers the
// elements [(c * 64 * W + r) * EL, + EL), EL = 16 bytes of elements.  Rows need only their
// element's alignment (H may be odd): global 16-byte loads and stores take any address.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "launch.h"

namespace moe {

template <typename T>
constexpr int kRowEl = 16 / (int)sizeof(T);   // uint16_t: bf16 bits; float: f32

// kVec: H is a multiple of EL, so a chunk is either whole or empty.
template <typename T, bool kVec>
__device__ __forceinline__ uint4 load_chunk(const T* p, int nvalid) {
  uint4 r = make_uint4(0, 0, 0, 0);
  if (kVec ? nvalid > 0 : nvalid >= kRowEl<T>) {
    __builtin_memcpy(&r, p, 16);
  } else if (!kVec && nvalid > 0) {
    T e[kRowEl<T>];
#pragma unroll
    for (int i = 0; i < kRowEl<T>; ++i) e[i] = i < nvalid ? p[i] : T(0);
    __builtin_memcpy(&r, e, 16);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void chunk_to_f32(const uint4& r, float (&v)[kRowEl<T>]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      v[i] = __uint_as_float(u[i]);
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 chunk_from_f32(const float (&v)[kRowEl<T>]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2)
      u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    else
      u[i] = __float_as_uint(v[i]);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// kNt: not kept in the caches
template <typename T, bool kVec, bool kNt = false>
__device__ __forceinline__ void store_chunk(T* p, const uint4& r, int nvalid) {
  if (kVec ? nvalid > 0 : nvalid >= kRowEl<T>) {
    typedef __attribute__((__vector_size__(16), __aligned__(2))) uint32_t AnyU32x4;
    if constexpr (kNt)
      __builtin_nontemporal_store(AnyU32x4{r.x, r.y, r.z, r.w}, reinterpret_cast<AnyU32x4*>(p));
    else
      __builtin_memcpy(p, &r, 16);
  } else if (!kVec && nvalid > 0) {
    T e[kRowEl<T>];
    __builtin_memcpy(e, &r, 16);
#pragma unroll
    for (int i = 0; i < kRowEl<T>; ++i)
      if (i < nvalid) p[i] = e[i];
  }
}

// n values of a parameter vector (bf16 or f32, element-aligned) as f32; absent entries and a
// null vector give `fill`
template <int n>
__device__ __forceinline__ void load_params(const void* p, bool bf16, long long at, int nvalid, float fill,
                                            float (&v)[n]) {
  if (p && nvalid >= n) {   // whole: n / 8 or n / 4 loads of 16 bytes (at least one of 8)
    if (bf16) {
      uint32_t u[n / 2];
      __builtin_memcpy(u, static_cast<const uint16_t*>(p) + at, 2 * n);
#pragma unroll
      for (int i = 0; i < n; ++i) v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    } else {
      __builtin_memcpy(v, static_cast<const float*>(p) + at, 4 * n);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float f = fill;
    if (p && i < nvalid)
      f = bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p)[at + i]) : static_cast<const float*>(p)[at + i];
    v[i] = f;
  }
}

// The sum over a row of 16 lanes of groups that repeat every `from` lanes: rotations, so that every
// lane adds the same values pairwise in the same tree and gets the same bits.
template <int from>
__device__ __forceinline__ float lanes16_sum(float v) {
  auto rotated = [](float x, auto by) {   // row_ror:by
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x120 + decltype(by)::value, 0xf, 0xf, false));
  };
  if constexpr (from >= 16) v += rotated(v, std::integral_constant<int, 8>{});
  if constexpr (from >= 8) v += rotated(v, std::integral_constant<int, 4>{});
  if constexpr (from >= 4) v += rotated(v, std::integral_constant<int, 2>{});
  if constexpr (from >= 2) v += rotated(v, std::integral_constant<int, 1>{});
  return v;
}

// The sum over the 64 lanes, in every lane (the same bits): within rows of 16 lanes, then across
// them by exchanging rows, without a trip through LDS.
__device__ __forceinline__ float wave_total(float v) {
  v = lanes16_sum<16>(v);
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Sums of N values over the W waves of a row; every lane gets them.  red: two buffers of kMaxSums
// floats per wave of the block; `buf` (0 or 1) alternates between consecutive calls, so that the
// barrier of the call in between separates a buffer's readers from its next writers, whatever N
// each call has.
constexpr int kMaxSums = 2;
template <int W, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int buf, int nwaves) {
  static_assert(N <= kMaxSums, "a buffer's floats per wave");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_total(v[i]);
  if constexpr (W > 1) {
    const int wave = threadIdx.x >> 6;
    float* mine = red + buf * nwaves * kMaxSums;
    if (lane_id() == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) mine[wave * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes16_sum<W>(mine[((wave / W) * W + lane_id() % W) * N + i]);
  }
}

// Waves per row and chunks per lane for `units` 16-byte units of a row: the fewest waves that
// hold it in at most kMaxC chunks a lane, or sixteen waves with up to kWideC, the widest row's.
template <typename T>
constexpr int kWideChunks = (int)(kNormMaxH / (16 * kWave * kRowEl<T>));

template <int kMaxC, int kWideC, int W, int C, typename F>
hipError_t dispatch_row_from(int u, F&& f) {
  if (u <= W * C) return f.template operator()<W, C>();
  if constexpr (W < 16 ? C < kMaxC : C < kWideC)
    return dispatch_row_from<kMaxC, kWideC, W, C + 1>(u, f);
  else if constexpr (W < 16)
    return dispatch_row_from<kMaxC, kWideC, 2 * W, C / 2 + 1>(u, f);
  return hipErrorInvalidValue;
}
template <int kMaxC, int kWideC, typename F>
hipError_t dispatch_row(int units, F&& f) {
  return dispatch_row_from<kMaxC, kWideC, 1, 1>((units + kWave - 1) / kWave, f);
}

}  // namespace moe
