// adamw.hip -- an AdamW step over many tensors (Loshchilov and Hutter, "Decoupled Weight Decay
// Regularization", ICLR 2019), with states in f32 or in e4m3 with a scale per 128 elements.
//
// With g = grad * grad_scale and t the step's number, per element:
//
//     m <- beta1 m + (1 - beta1) g,   v <- beta2 v + (1 - beta2) g^2
//     p <- p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// The step is bound by HBM: an element of bf16 parameters with bf16 gradients moves 22 bytes with
// f32 states and 10 with 8-bit ones.  With f32 states, an f32 copy and f32 gradients 75 million elements take
// 500 us, 4.5 TB/s (a copy of as many bytes runs at 4.8 to 5.1); with 8-bit states and rounding by chance 100
// million elements take 224 to 231 us one call after the other, 4.4 TB/s, with the VALU busy for most of it (94
// instructions an element).  By the profiler's durations, with its pauses between the calls, 499 to 507 and 225 to 266 us
// (least and median of 15).
// A lane therefore takes 8 consecutive elements, so that every access is 8 or 16 bytes a lane and 16 lanes hold
// a block of 128 elements: the block's largest value is a reduction over 16 lanes by rotations, without LDS.
// A workgroup takes 2048 elements of one tensor, found by a binary search over the first workgroups of up to 64
// tensors that travel in the
// kernel's arguments: one launch for 64 tensors, nothing to copy or allocate.
//
// 8-bit states hold m and sqrt(v), not v: the root halves the exponents' range, so that e4m3's
// 2^-9 to 448 covers v over 2^35 within a block, and a value above zero never rounds to the code of zero (its
// update would divide by eps).  Rounding to nearest would freeze a slow average: beta2 = 0.999 moves sqrt(v)
// by at most 0.05% a step, a code's step is 6 to 12%.  With rng the codes (and bf16 parameters without an f32
// copy) are rounded up with the chance of the remainder instead, by 16 bits of Philox4x32-10 (the dropout's
// generator) for each element, one of eight in a counter block.  m, v and p share an element's bits: each is
// unbiased by itself.
//
// The arithmetic is single operations, each rounded once (no contraction), so that a plain
// evaluation in f32 in the same order takes the same rounding decisions.

#include <math.h>

#include "dropout_device.h"
#include "launch.h"
#include "rows_device.h"

namespace moe {

namespace {

constexpr int kPer = 8;                      // elements a lane
constexpr int kThreads = 256;
constexpr int kChunk = kThreads * kPer;      // elements a workgroup
constexpr int kTensors = 64;                 // tensors of a launch
constexpr uint32_t kStream = 2;              // counter word 2: apart from the dropout's 0 and 1

struct Slot {
  void* p;
  const void* g;
  long long n;
  long long start;   // first element in the state arrays
};

struct Args {
  Slot slot[kTensors];
  int first[kTensors + 1];   // first workgroup of each tensor; the launch's count
  int count;
  void *m, *v;
  float *m_scale, *v_scale;
  float* master;
  float beta1, rest1, beta2, rest2, eps;
  float decay, step_size, root;   // 1 - lr wd, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  float weight_decay;
  const float* schedule;          // lr, 1 - beta1^t, 1 - beta2^t, in place of the three above
  const float* grad_scale;
  const uint64_t* rng;
};

// bits 16 (j & 1) on of word j / 2: the 16-bit piece of element j of a counter block
__device__ __forceinline__ uint32_t piece16(const uint4& r, int j) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  return (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
}

// e4m3 code of x, |x| <= 448 (1 + 2^-22), rounded up in magnitude with the chance of the remainder: the
// mantissa bits below e4m3's three are a 20-bit fraction of a step, and the piece, centred in its
// share of 16, is added to them.  Codes below the smallest normal (2^-6) have its step, so 2^-6 is added to
// round there and taken off the code.
//
// No branches here: a lane's early return for each of 16 values took as many instructions as the rounding.
template <bool kSigned, bool kFinite>
__device__ __forceinline__ uint32_t e4m3_by_chance(float x, uint32_t piece) {
  const float a = fabsf(x);
  const bool small = a < 0.015625f;
  const uint32_t b = __float_as_uint(small ? a + 0.015625f : a) + (piece << 4) +
                     (small ? 8u - (968u << 20) : 8u - (960u << 20));
  uint32_t code = min(b >> 20, 126u);
  if (kSigned) code |= (__float_as_uint(x) >> 24) & 0x80u;
  return kFinite || a < INFINITY ? code : 0x7fu;
}

// 8 codes of a block of 128 elements (16 lanes): scale = amax * (1 / 448).  kLeast: no value is negative, and those
// above zero keep code 1.  kFinite: there are no infinities or NaN.
template <bool kLeast, bool kFinite>
__device__ __forceinline__ uint2 pack_block(const float (&x)[kPer], const uint4& bits, bool chance, float& scale) {
#pragma clang fp contract(off)
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) amax = fmaxf(amax, fabsf(x[j]));   // without NaN: the codes keep those
  auto rotated = [](float f, auto by) {   // row_ror:by
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(f), 0x120 + decltype(by)::value, 0xf, 0xf, false));
  };
  amax = fmaxf(amax, rotated(amax, std::integral_constant<int, 8>{}));
  amax = fmaxf(amax, rotated(amax, std::integral_constant<int, 4>{}));
  amax = fmaxf(amax, rotated(amax, std::integral_constant<int, 2>{}));
  amax = fmaxf(amax, rotated(amax, std::integral_constant<int, 1>{}));
  const bool some = amax >= 0x1p-100f;   // below: zeros (1 / amax is finite above)
  scale = some ? amax * (1.0f / 448.0f) : 1.0f;
  const float inv = some ? 448.0f * (1.0f / amax) : 0.0f;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < kPer; j += 2) {
    const float a = x[j] * inv, b = x[j + 1] * inv;
    const uint32_t la = kLeast && x[j] > 0.0f && some ? 1u : 0u, lb = kLeast && x[j + 1] > 0.0f && some ? 1u : 0u;
    uint32_t c;
    if (chance) {
      c = max(e4m3_by_chance<!kLeast, kFinite>(a, piece16(bits, j)), la) |
          max(e4m3_by_chance<!kLeast, kFinite>(b, piece16(bits, j + 1)), lb) << 8;
    } else {
      c = cvt_e4m3x2(a, b);
      if (kLeast) c = max(c & 0xffu, la) | max(c >> 8 & 0xffu, lb) << 8;
    }
    w[j >> 2] |= c << (8 * (j & 2));
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void unpack_block(const uint2& c, float scale, float (&x)[kPer]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    x[4 * h] = __builtin_amdgcn_cvt_f32_fp8(w[h], 0) * scale;
    x[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(w[h], 1) * scale;
    x[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(w[h], 2) * scale;
    x[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(w[h], 3) * scale;
  }
}

// 8 elements of a tensor as f32 (zeros past its end); at is a multiple of 8, so whole pieces are aligned
template <typename T>
__device__ __forceinline__ void load8(const void* p, long long at, int n, float (&x)[kPer]) {
  const T* q = static_cast<const T*>(p) + at;
  if constexpr (sizeof(T) == 2) {
    chunk_to_f32<T>(load_chunk<T, false>(q, n), x);
  } else {
    float lo[4], hi[4];
    chunk_to_f32<T>(load_chunk<T, false>(q, n), lo);
    chunk_to_f32<T>(load_chunk<T, false>(q + 4, n - 4), hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = lo[j];
      x[4 + j] = hi[j];
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(void* p, long long at, int n, const float (&x)[kPer]) {
  T* q = static_cast<T*>(p) + at;
  if constexpr (sizeof(T) == 2) {
    store_chunk<T, false>(q, chunk_from_f32<T>(x), n);
  } else {
    const float lo[4] = {x[0], x[1], x[2], x[3]}, hi[4] = {x[4], x[5], x[6], x[7]};
    store_chunk<T, false>(q, chunk_from_f32<T>(lo), n);
    store_chunk<T, false>(q + 4, chunk_from_f32<T>(hi), n - 4);
  }
}

// u = sqrt(v), rounded to nearest.  Goldschmidt's iteration on a 1-ulp reciprocal root and Markstein's last
// correction by the residual take 10 instructions for sqrtf's 16.  The residual v - s^2 is a multiple of 2^-48 v and
// has to be exact: from v = 2^-96 on it is, as a subnormal number in part.  A wave with a smaller v above zero, or with
// one that is negative, infinite or NaN, takes sqrtf: the clamp below would make numbers of a root that is NaN.
__device__ __forceinline__ void roots(const float (&v)[kPer], float (&u)[kPer]) {
#pragma clang fp contract(off)
  uint32_t least = 0xffffffffu, most = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    least = min(least, __float_as_uint(v[j]) - 1u);   // zeros pass
    most = max(most, __float_as_uint(v[j]));          // with a sign, or infinite, or NaN: from 0x7f800000 on
  }
  if (__any(least < 0x0f800000u - 1u || most >= 0x7f800000u)) {   // 2^-96
#pragma unroll
    for (int j = 0; j < kPer; ++j) u[j] = sqrtf(v[j]);
    return;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float y = fminf(__builtin_amdgcn_rsqf(v[j]), 0x1p60f);   // of zero: its products with zero are zeros
    float s = v[j] * y, h = 0.5f * y;
    const float e = fmaf(-s, h, 0.5f);
    s = fmaf(s, e, s);
    h = fmaf(h, e, h);
    u[j] = fmaf(fmaf(-s, s, v[j]), h, s);
  }
}

template <typename P, typename G, bool S8, bool MASTER>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Args a) {
#pragma clang fp contract(off)
  int lo = 0, hi = a.count;   // largest tensor whose first workgroup is not past this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= (int)blockIdx.x) lo = mid; else hi = mid;
  }
  const Slot s = a.slot[lo];
  const long long at = (long long)((int)blockIdx.x - a.first[lo]) * kChunk + threadIdx.x * kPer;
  // whole blocks of the states: lanes past the tensor's last block have nothing (16 lanes at a time)
  if (at >= ((s.n + 127) & ~127ll)) return;
  const int n = (int)max(0ll, min((long long)kPer, s.n - at));
  const long long sat = s.start + at;

  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  if (!(fabsf(gs) < INFINITY)) return;   // uniform: a step without a usable gradient changes nothing

  float p[kPer], g[kPer], m[kPer], v[kPer];
  load8<G>(s.g, at, n, g);
  if constexpr (MASTER) load8<float>(a.master, sat, n, p); else load8<P>(s.p, at, n, p);
  if constexpr (S8) {
    const uint2 cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.m) + sat);
    const uint2 cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.v) + sat);
    unpack_block(cm, a.m_scale[sat >> 7], m);
    unpack_block(cv, a.v_scale[sat >> 7], v);
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = v[j] * v[j];
  } else {
    load8<float>(a.m, sat, n, m);
    load8<float>(a.v, sat, n, v);
  }
  float decay = a.decay, step_size = a.step_size, root = a.root;
  if (a.schedule) {
    const float lr = a.schedule[0];
    decay = 1.0f - lr * a.weight_decay;
    step_size = lr / a.schedule[1];
    root = 1.0f / sqrtf(a.schedule[2]);
  }
  float u[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float gj = g[j] * gs;
    m[j] = m[j] * a.beta1 + gj * a.rest1;
    v[j] = v[j] * a.beta2 + (gj * gj) * a.rest2;
  }
  roots(v, u);
  float all = 0.0f;   // finite only if every result is
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float upd = m[j] / (u[j] * root + a.eps);
    p[j] = p[j] * decay - upd * step_size;
    all += fabsf(p[j]) + (S8 ? fabsf(m[j]) + u[j] : 0.0f);
  }
  const bool finite = !__any(!(all < INFINITY));   // uniform: the few cases of infinities and NaN apart
  if (S8 && n < kPer) {   // the rest of a tensor's last block
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j >= n) m[j] = u[j] = 0.0f;
  }
  uint4 bits = make_uint4(0, 0, 0, 0);
  const bool chance = a.rng != nullptr;
  if (chance) bits = philox4x32(a.rng[1] + (uint64_t)(sat >> 3), kStream, a.rng[0]);
  if constexpr (MASTER) store8<float>(a.master, sat, n, p);
  if (sizeof(P) == 2 && !MASTER && chance) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t b = __float_as_uint(p[j]);
      w[j >> 1] |= (b + piece16(bits, j)) >> 16 << (16 * (j & 1));
    }
    if (!finite) {   // infinities and NaN keep their upper half (a NaN its quiet bit)
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (fabsf(p[j]) < INFINITY) continue;
        const uint32_t b = __float_as_uint(p[j]) | (p[j] == p[j] ? 0u : 0x400000u);
        w[j >> 1] = (w[j >> 1] & 0xffffu << (16 - 16 * (j & 1))) | b >> 16 << (16 * (j & 1));
      }
    }
    store_chunk<uint16_t, false>(static_cast<uint16_t*>(s.p) + at, make_uint4(w[0], w[1], w[2], w[3]), n);
  } else {
    store8<P>(s.p, at, n, p);
  }
  if constexpr (S8) {
    float sm, sv;
    uint2 cm, cv;
    if (finite) {
      cm = pack_block<false, true>(m, bits, chance, sm);
      cv = pack_block<true, true>(u, bits, chance, sv);
    } else {
      cm = pack_block<false, false>(m, bits, chance, sm);
      cv = pack_block<true, false>(u, bits, chance, sv);
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + sat) = cm;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + sat) = cv;
    if ((threadIdx.x & 15) == 0) {
      a.m_scale[sat >> 7] = sm;
      a.v_scale[sat >> 7] = sv;
    }
  } else {
    store8<float>(a.m, sat, n, m);
    store8<float>(a.v, sat, n, v);
  }
}

template <typename P, typename G, bool S8, bool MASTER>
hipError_t launch(const Args& a, hipStream_t stream) {
  hipLaunchKernelGGL((adamw_kernel<P, G, S8, MASTER>), dim3(a.first[a.count]), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename P, typename G>
hipError_t launch_states(const Args& a, bool s8, hipStream_t stream) {
  if constexpr (sizeof(P) == 2)
    if (a.master) return s8 ? launch<P, G, true, true>(a, stream) : launch<P, G, false, true>(a, stream);
  return s8 ? launch<P, G, true, false>(a, stream) : launch<P, G, false, false>(a, stream);
}

}  // namespace

hipError_t launch_adamw(const AdamwLaunch& q, hipStream_t stream) {
  Args a{};
  a.m = q.m;
  a.v = q.v;
  a.m_scale = q.m_scale;
  a.v_scale = q.v_scale;
  a.master = q.master;
  a.beta1 = (float)q.beta1;
  a.rest1 = (float)(1.0 - q.beta1);
  a.beta2 = (float)q.beta2;
  a.rest2 = (float)(1.0 - q.beta2);
  a.eps = (float)q.eps;
  a.weight_decay = (float)q.weight_decay;
  a.decay = (float)(1.0 - q.lr * q.weight_decay);
  a.step_size = (float)(q.lr / (1.0 - pow(q.beta1, (double)q.step)));
  a.root = (float)(1.0 / sqrt(1.0 - pow(q.beta2, (double)q.step)));
  a.schedule = q.schedule;
  a.grad_scale = q.grad_scale;
  a.rng = q.rng;
  long long start = 0, blocks = 0;
  hipError_t e = hipSuccess;
  auto flush = [&]() {
    if (!a.count) return;
    a.first[a.count] = (int)blocks;
    if (q.p_bf16)
      e = q.g_bf16 ? launch_states<uint16_t, uint16_t>(a, q.s8, stream) : launch_states<uint16_t, float>(a, q.s8, stream);
    else
      e = q.g_bf16 ? launch_states<float, uint16_t>(a, q.s8, stream) : launch_states<float, float>(a, q.s8, stream);
    a.count = 0;
    blocks = 0;
  };
  for (long long i = 0; i < q.count && e == hipSuccess; ++i) {
    const long long n = q.n[i];
    if (n > 0) {
      const long long mine = (n + kChunk - 1) / kChunk;
      if (a.count == kTensors || blocks + mine >= (1ll << 32) / kThreads) flush();   // n <= 2^34
      a.slot[a.count] = Slot{q.param[i], q.grad[i], n, start};
      a.first[a.count++] = (int)blocks;
      blocks += mine;
    }
    start += (n + 127) & ~127ll;
  }
  if (e == hipSuccess) flush();
  return e;
}

}  // namespace moe
