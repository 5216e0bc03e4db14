// rows_device.h -- reading and writing token rows 16 bytes a lane, and sums over the waves of a row.
//
// A row of H elements is held by W waves with C chunks a lane: chunk c of row lane r covers the
// elements [(c * 64 * W + r) * EL, + EL), EL = 16 bytes of elements.  Rows need only their
// element's alignment (H may be odd): global 16-byte loads and stores take any address.
#pragma once

#include "device_common.h"

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

template <typename T, bool kVec>
__device__ __forceinline__ void store_chunk(T* p, const uint4& r, int nvalid) {
  if (kVec ? nvalid > 0 : nvalid >= kRowEl<T>) {
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
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float f = fill;
    if (p && i < nvalid)
      f = bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p)[at + i]) : static_cast<const float*>(p)[at + i];
    v[i] = f;
  }
}

// Sums of a and b over the W waves of a row; every lane gets them.  red: 2 * waves-per-block
// pairs of LDS; `buf` (0 or 1) alternates between consecutive calls, so that the barrier of the
// call in between separates a buffer's readers from its next writers.
template <int W>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2* red, int buf, int nwaves) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (W > 1) {
    const int wave = threadIdx.x >> 6;
    if (lane_id() == 0) red[buf * nwaves + wave] = make_float2(a, b);
    __syncthreads();
    a = 0.0f;
    b = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 s = red[buf * nwaves + (wave / W) * W + i];
      a += s.x;
      b += s.y;
    }
  }
}

// waves per row and chunks per lane for `units` 16-byte units of a row: the fewest waves that
// hold it in at most four chunks a lane (eight at sixteen waves)
template <typename F>
inline hipError_t dispatch_row(int units, F&& f) {
  const int u = (units + kWave - 1) / kWave;
  if (u <= 1) return f.template operator()<1, 1>();
  if (u <= 2) return f.template operator()<1, 2>();
  if (u <= 3) return f.template operator()<1, 3>();
  if (u <= 4) return f.template operator()<1, 4>();
  if (u <= 6) return f.template operator()<2, 3>();
  if (u <= 8) return f.template operator()<2, 4>();
  if (u <= 12) return f.template operator()<4, 3>();
  if (u <= 16) return f.template operator()<4, 4>();
  if (u <= 24) return f.template operator()<8, 3>();
  if (u <= 32) return f.template operator()<8, 4>();
  if (u <= 64) return f.template operator()<16, 4>();
  return f.template operator()<16, 8>();
}

}  // namespace moe
