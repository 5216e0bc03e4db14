// decode.hip -- the whole expert layer for up to 16 tokens in two kernels:
//
//   up:    route each token, h[r] = silu(W13_gate[e] x_t) * (W13_up[e] x_t) for each routed row r = t k + j
//   down:  out[t] = sum over j of weight[r] * (W2[e] h[r]), j ascending
//
// on bf16 weights, 8-bit integers with a scale per output channel, e4m3 with a scale per 128 x 128 block, int4
// with f32 scales per 32, 64 or 128 channels, or mxfp4.  Activations stay in bf16: weights are turned into bf16
// operands in registers, where all of these codes are exact, and scales multiply f32 sums (mxfp4's
// powers of two the operand).
//
// The bytes of the routed experts' weights bound it: every weight is read once, straight into registers, a
// few 128-byte pieces of 16 weight rows ahead in each wave.  The 16 tokens' side of
// v_mfma_f32_16x16x32_bf16 takes an expert's tokens, as many as there are: one token costs what 16 do.
// Activations come from the caches in the same order as the weights, so that the wait for
// a piece's weights is the wait for its activations too.
//
// The routing is recomputed by each workgroup of the first kernel (a wave a token at a time; a third launch or
// a wait between workgroups would cost more) and left for the second one.  In the first a
// workgroup's four waves share K of 16 columns (16 gate and 16 up rows) of one expert; in the second eight
// waves share all experts' K of 16 output columns, so that a token's sum over its experts ends in one place
// and needs no atomics: sums are joined through LDS in a fixed order.

#include <algorithm>

#include "decode_plan.h"
#include "fourbit_device.h"
#include "launch.h"
#include "route_device.h"

namespace moe {

namespace {

enum Fmt { kBf16, kInt8, kE4m3, kInt4x32, kInt4x64, kInt4x128, kMxfp4 };

template <int F>
struct FmtOf {
  static constexpr bool kInt4 = F == kInt4x32 || F == kInt4x64 || F == kInt4x128;
  static constexpr bool kFour = kInt4 || F == kMxfp4;
  static constexpr int kBits = F == kBf16 ? 16 : kFour ? 4 : 8;
  static constexpr int kVal = 128 / kBits;            // weights in 16 bytes
  static constexpr int kX = kVal / 8;                 // 16-byte pieces of activations for them
  static constexpr int kGroup = F == kInt4x32 || F == kMxfp4 ? 32 : F == kInt4x64 ? 64 : 128;
  // 64-byte pieces of a weight row in a step: four lanes' 16 bytes, once or twice
  static constexpr int kPieces = kFour ? 1 : 2;
  static constexpr int kStep = 64 * kPieces;
  static constexpr int kGroups = kInt4 ? std::max(1, 64 * 2 / kGroup) : 1;   // int4 scales of a step
};

// one step's weights, activations and scales of a lane
template <int F, int NM>
struct Step {
  using T = FmtOf<F>;
  uint4 w[NM][T::kPieces];
  uint4 x[T::kPieces][T::kX];
  uint32_t s[NM][T::kGroups];   // bits of int4's f32 scales or e4m3's block scale, or mxfp4's byte
};

// 16 bytes, or zeros
__device__ __forceinline__ uint4 load_if(bool live, const uint8_t* p) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (live) v = *reinterpret_cast<const uint4*>(p);
  return v;
}

// four signed bytes as bf16
__device__ __forceinline__ uint2 unpack_int8(uint32_t v) {
  const float a = (float)(int8_t)v, b = (float)(int8_t)(v >> 8), c = (float)(int8_t)(v >> 16), d = (float)(int8_t)(v >> 24);
  return make_uint2(__builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u),
                    __builtin_amdgcn_perm(__float_as_uint(d), __float_as_uint(c), 0x07060302u));
}

__device__ __forceinline__ uint2 unpack_e4m3(uint32_t v) {
  return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true)));
}

template <int F>
__device__ __forceinline__ bf16x8 unpack8(uint32_t lo, uint32_t hi) {   // 8 codes of 8 bits
  const uint2 a = F == kInt8 ? unpack_int8(lo) : unpack_e4m3(lo), b = F == kInt8 ? unpack_int8(hi) : unpack_e4m3(hi);
  return as_bf16x8(make_uint4(a.x, a.y, b.x, b.y));
}

// NM weight rows' products with an expert's tokens over the steps of a wave: units of 128 bytes of
// the rows, first, first + stride, ...
//
// MFMA layout: the lane's weight row is column lane % 16 of the result, the lane's token row row
// lane % 16 of the activations; lane / 16 = g picks the lane's 16 bytes of a 64-byte piece.  acc[m][r]
// becomes the sum of token 4 g + r and the lane's weight row.  int4: after a transpose of
// words between the lane groups each MFMA has 32 consecutive channels, so activations are read to fit that.
//
// Addresses are a scalar base that walks along the row and a 32-bit offset of the lane that stays: three
// vector registers for all streams.
template <int F, int NM, int DEPTH>
struct Products {
  using T = FmtOf<F>;
  const uint8_t* w[NM];      // uniform: the expert's first weight row
  uint32_t w_off;            // the lane's row, and 16 g
  const uint8_t* x;          // uniform
  uint32_t x_off;            // the lane's token row, and its channels of a piece
  const uint8_t* s[NM];      // uniform
  uint32_t s_off;            // int4, mxfp4: the lane's row (mxfp4: and g)
  int row_bytes;             // of a weight row
  int g;

  static __device__ __forceinline__ uint32_t x_lane(int g) { return T::kInt4 ? 16 * g : 16 * T::kX * g; }

  template <bool WHOLE>
  __device__ __forceinline__ void load(Step<F, NM>& b, int at) const {
    const uint8_t* xs = x + (long long)(at / 16) * (T::kVal * 2);
#pragma unroll
    for (int p = 0; p < T::kPieces; ++p) {
      const bool live = WHOLE || at + 64 * p + 16 * g < row_bytes;
#pragma unroll
      for (int q = 0; q < T::kX; ++q) {
        // int4: the lane's 8 channels of the q-th 32; else the q-th 8 of its own piece's
        const uint8_t* from = xs + (T::kInt4 ? 64 * q : 64 * T::kX * p + 16 * q);
        b.x[p][q] = load_if(T::kInt4 ? WHOLE || at + 16 * q < row_bytes : live, from + x_off);
      }
#pragma unroll
      for (int m = 0; m < NM; ++m)
        b.w[m][p] = load_if(live, w[m] + at + 64 * p + w_off);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      if constexpr (F == kE4m3) b.s[m][0] = *reinterpret_cast<const uint32_t*>(s[m] + (at >> 7) * 4);
      if constexpr (F == kMxfp4) {
        b.s[m][0] = 0;
        if (WHOLE || at + 16 * g < row_bytes) b.s[m][0] = *(s[m] + (at >> 4) + s_off);
      }
      if constexpr (T::kInt4) {
        const uint8_t* from = s[m] + at * 2 / T::kGroup * 4;
        if constexpr (WHOLE) {
          __builtin_memcpy(b.s[m], from + s_off, 4 * T::kGroups);
        } else {
#pragma unroll
          for (int q = 0; q < T::kGroups; ++q) {
            b.s[m][q] = 0;
            if (at + q * (T::kGroup / 2) < row_bytes) __builtin_memcpy(&b.s[m][q], from + 4 * q + s_off, 4);
          }
        }
      }
    }
  }

  static __device__ __forceinline__ void use(const Step<F, NM>& b, f32x4 (&acc)[NM]) {
    if constexpr (F == kBf16) {
#pragma unroll
      for (int p = 0; p < T::kPieces; ++p)
#pragma unroll
        for (int m = 0; m < NM; ++m)
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(b.x[p][0]), as_bf16x8(b.w[m][p]), acc[m], 0, 0, 0);
    } else if constexpr (F == kInt8 || F == kE4m3) {
      f32x4 part[NM];
#pragma unroll
      for (int m = 0; m < NM; ++m) part[m] = F == kE4m3 ? f32x4{0, 0, 0, 0} : acc[m];
#pragma unroll
      for (int p = 0; p < T::kPieces; ++p)
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          const uint4 v = b.w[m][p];
          part[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(b.x[p][0]), unpack8<F>(v.x, v.y), part[m], 0, 0, 0);
          part[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(b.x[p][1]), unpack8<F>(v.z, v.w), part[m], 0, 0, 0);
        }
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[m][r] = F == kE4m3 ? fmaf(part[m][r], __uint_as_float(b.s[m][0]), acc[m][r]) : part[m][r];
    } else if constexpr (F == kMxfp4) {
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const uint4 v = b.w[m][0];
        const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(b.x[0][q]), as_bf16x8(unpack_mxfp4(d[q], b.s[m][0])),
                                                           acc[m], 0, 0, 0);
      }
    } else {
      uint32_t d[NM][4];
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const uint4 v = b.w[m][0];
        d[m][0] = v.x, d[m][1] = v.y, d[m][2] = v.z, d[m][3] = v.w;
        transpose4(d[m]);
      }
      // a group's sum of code * x starts from -8 * sum of x
      const bf16x8 minus8 = as_bf16x8(make_uint4(0xc100c100u, 0xc100c100u, 0xc100c100u, 0xc100c100u));
      constexpr int kPer = 4 / T::kGroups;   // MFMAs of a scale
#pragma unroll
      for (int q0 = 0; q0 < 4; q0 += kPer) {
        f32x4 part[NM];
#pragma unroll
        for (int q = q0; q < q0 + kPer; ++q) {
          const bf16x8 xo = as_bf16x8(order_int4(b.x[0][q]));
          const f32x4 start = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, minus8, f32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            const f32x4 one = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, as_bf16x8(unpack_int4(d[m][q])), start, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) part[m][r] = q == q0 ? one[r] : part[m][r] + one[r];
          }
        }
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][r] = fmaf(part[m][r], __uint_as_float(b.s[m][q0 / kPer]), acc[m][r]);
      }
    }
  }

  // steps of a share: units first, first + stride, ... of a row
  static __device__ __forceinline__ int steps(int row_bytes, int first, int stride) {
    const int units = (row_bytes + 127) >> 7;
    const int n = first < units ? (units - first + stride - 1) / stride : 0;
    if constexpr (T::kPieces == 2) return n;
    const bool half = n > 0 && first + (n - 1) * stride == units - 1 && row_bytes <= units * 128 - 64;
    return 2 * n - (half ? 1 : 0);
  }
};

// Streams the products of jobs 0 to jobs - 1 through a wave: the loads run DEPTH steps ahead of the MFMAs, across the
// ends of jobs.  start(job, products, first, stride) sets a job's streams and its share of K, steps_of(job)
// is the number of its steps (at least one), finish(job, sums) takes its sums.
template <int F, int NM, int DEPTH, typename Start, typename Steps, typename Finish>
__device__ __forceinline__ void stream(int jobs, Start&& start, Steps&& steps_of, Finish&& finish) {
  using P = Products<F, NM, DEPTH>;
  using T = FmtOf<F>;
  if (jobs <= 0) return;
  P p;
  int first = 0, stride = 1, load_job = 0, load_step = 0;
  start(0, p, first, stride);
  int load_steps = steps_of(0);
  int use_job = 0, left = load_steps;   // of the job in use
  auto get = [&](Step<F, NM>& b) {
    if (load_job >= jobs) return;
    const int at = T::kPieces == 2 ? (first + load_step * stride) * 128
                                   : (first + (load_step >> 1) * stride) * 128 + (load_step & 1) * 64;
    if (at + T::kStep <= p.row_bytes)
      p.template load<true>(b, at);
    else
      p.template load<false>(b, at);
    if (++load_step == load_steps) {
      load_step = 0;
      if (++load_job < jobs) {
        start(load_job, p, first, stride);
        load_steps = steps_of(load_job);
      }
    }
  };
  Step<F, NM> b[DEPTH];
  f32x4 acc[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) acc[m] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < DEPTH; ++j) get(b[j]);
  while (true) {
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) {
      P::use(b[j], acc);
      get(b[j]);
      if (--left == 0) {
        finish(use_job, acc);
        if (++use_job == jobs) return;
        left = steps_of(use_job);
#pragma unroll
        for (int m = 0; m < NM; ++m) acc[m] = f32x4{0, 0, 0, 0};
      }
    }
  }
}

template <int F>
constexpr int kDepthUp = FmtOf<F>::kInt4 || F == kE4m3 ? 2 : 3;
template <int F>
constexpr int kDepthDown = FmtOf<F>::kInt4 || F == kE4m3 ? 3 : 4;
// workgroups on a CU that the registers leave room for
template <int F>
constexpr int kUpGroups = F == kInt4x32 ? 3 : 4;

constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;
constexpr int kDownParts = 768;   // routed rows times shares of K that the second kernel's LDS holds

struct UpArgs {
  const uint8_t* x;       // [T, H] bf16
  const float* logits;    // [T, E]
  const uint8_t* w;       // [E, 2I, H]
  const uint8_t* s;
  int T, H, I, E, k, valid, renorm;
  int blocks;             // ceil(I / 16)
  DecodePlan* plan;
  uint16_t* h;            // [T k, I] bf16
};

// bytes of the scales of a weight row of K channels (e4m3: of a row of blocks)
template <int F>
__device__ __forceinline__ int scale_bytes(int K) {
  if constexpr (F == kE4m3) return K / 128 * 4;
  if constexpr (F == kMxfp4) return K / 32;
  if constexpr (FmtOf<F>::kInt4) return K / FmtOf<F>::kGroup * 4;
  return 0;
}

// the streams of a wave whose lanes' weight rows are base + n, n below 2^32 bytes of weights on
template <int F, int NM, int DEPTH>
__device__ __forceinline__ void set_rows(Products<F, NM, DEPTH>& p, const uint8_t* w, const uint8_t* s,
                                         const long long (&base)[NM], int n0, int n, int K) {
  const int g = lane_id() >> 4, sb = scale_bytes<F>(K);
  p.g = g;
  p.row_bytes = K / FmtOf<F>::kVal * 16;
  p.w_off = (uint32_t)n * (uint32_t)p.row_bytes + 16 * g;
  p.s_off = (uint32_t)n * (uint32_t)sb + (F == kMxfp4 ? g : 0);
#pragma unroll
  for (int m = 0; m < NM; ++m) {
    p.w[m] = w + base[m] * p.row_bytes;
    // e4m3: the block row of columns n0 to n0 + 15
    p.s[m] = F == kE4m3 ? s + ((base[m] + n0) >> 7) * sb : s + base[m] * sb;
  }
}

// Routes the tokens and lists the experts that have rows, in the order of their first row, with their
// rows in ascending order.  `words`: E, of LDS, twice.
template <int EPL>
__device__ __forceinline__ void make_plan(const UpArgs& a, DecodePlan& plan, uint32_t* tokens, uint32_t* index, int* ids) {
  const int wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < a.E; e += kUpWaves * kWave) tokens[e] = 0;
  for (int t = wave; t < a.T; t += kUpWaves)
    route_token<EPL>(a.logits, t, a.E, a.k, a.valid, a.renorm, ids, plan.weight);
  __syncthreads();
  const int r = threadIdx.x;   // T k <= 256
  const int e = r < a.T * a.k ? ids[r] : a.E;
  const int t = r / a.k;
  const bool live = (unsigned)e < (unsigned)a.E;
  if (live) atomicOr(&tokens[e], 1u << t);
  __syncthreads();
  const uint32_t mine = live ? tokens[e] : 0;
  const int rank = __popc(mine & ((1u << t) - 1));
  const bool first = live && rank == 0;
  // position among the first rows of experts: this wave's by ballot, the waves' by LDS
  const uint64_t firsts = __ballot(first);
  if (lane_id() == 0) ids[kDecodeRows + wave] = __popcll(firsts);
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kUpWaves; ++i) {
    const int n = ids[kDecodeRows + i];
    before += i < wave ? n : 0;
    all += n;
  }
  if (first) {
    const int at = before + __popcll(firsts & ((1ull << lane_id()) - 1));
    index[e] = at;
    plan.expert[at] = (uint16_t)e;
    plan.count[at] = (uint8_t)__popc(mine);
  }
  if (threadIdx.x == 0) plan.active = all;
  __syncthreads();
  if (live) plan.rows[index[e]][rank] = (uint8_t)r;
  __syncthreads();
}

template <int F, int EPL>
__global__ __launch_bounds__(kUpWaves * kWave, kUpGroups<F>) void decode_up_kernel(UpArgs a) {
  using T = FmtOf<F>;
  __shared__ DecodePlan plan;
  __shared__ uint32_t tokens[EPL * kWave], index[EPL * kWave];
  __shared__ int ids[kDecodeRows + kUpWaves];
  __shared__ float part[kUpWaves][2][16][17];
  make_plan<EPL>(a, plan, tokens, index, ids);
  if (blockIdx.x == 0) {   // for the second kernel
    const uint4* from = reinterpret_cast<const uint4*>(&plan);
    for (int i = threadIdx.x; i < (int)(sizeof(DecodePlan) / 16); i += kUpWaves * kWave)
      reinterpret_cast<uint4*>(a.plan)[i] = from[i];
  }
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int active = __builtin_amdgcn_readfirstlane(plan.active);
  const int items = active * a.blocks;   // (expert, 16 columns): blockIdx.x, + gridDim.x, ...
  const int jobs = items > (int)blockIdx.x ? (items - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;
  auto item_of = [&](int job, int& at, int& n0) {
    const int item = (int)blockIdx.x + job * (int)gridDim.x;
    at = item / a.blocks;
    n0 = (item - at * a.blocks) * 16;
  };
  const int steps = Products<F, 2, 1>::steps(a.H / T::kVal * 16, wave, kUpWaves);
  // the waves' sums of an item: joined by every thread for one token and column
  auto finish = [&](int job, const f32x4 (&acc)[2]) {
    int at, n0;
    item_of(job, at, n0);
    const int count = plan.count[at];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][m][4 * (lane >> 4) + r][lane & 15] = acc[m][r];
    __syncthreads();
    const int j = threadIdx.x >> 4, c = n0 + (threadIdx.x & 15);
    if (j < count && c < a.I) {
      float v[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        v[m] = 0.0f;
#pragma unroll
        for (int i = 0; i < kUpWaves; ++i) v[m] += part[i][m][j][threadIdx.x & 15];
        if (F == kInt8)
          v[m] *= reinterpret_cast<const float*>(a.s)[(long long)plan.expert[at] * 2 * a.I + m * a.I + c];
      }
      a.h[(long long)plan.rows[at][j] * a.I + c] = f32_to_bf16_bits(silu_mul(v[0], v[1]));
    }
    __syncthreads();
  };
  if (steps == 0) {   // a row of fewer units than waves: nothing to add
    const f32x4 none[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
    for (int job = 0; job < jobs; ++job) finish(job, none);
    return;
  }
  stream<F, 2, kDepthUp<F>>(
      jobs,
      [&](int job, auto& p, int& first, int& stride) {
        int at, n0;
        item_of(job, at, n0);
        const int e = __builtin_amdgcn_readfirstlane(plan.expert[at]), count = plan.count[at];
        const long long row = (long long)e * 2 * a.I;
        // columns past I repeat the last one, tokens past the expert's its last
        set_rows(p, a.w, a.s, {row, row + a.I}, n0, min(n0 + (lane & 15), a.I - 1), a.H);
        p.x = a.x;
        p.x_off = (uint32_t)(plan.rows[at][min(lane & 15, count - 1)] / a.k) * (uint32_t)a.H * 2 + p.x_lane(p.g);
        first = wave;
        stride = kUpWaves;
      },
      [&](int) { return steps; }, finish);
}

struct DownArgs {
  const DecodePlan* plan;
  const uint16_t* h;   // [T k, I] bf16
  const uint8_t* w;    // [E, H, I]
  const uint8_t* s;
  int T, H, I, k, valid;
  void* out;           // [T, H]
  int out_bf16;
};

template <int F>
__global__ __launch_bounds__(kDownWaves * kWave, 4) void decode_down_kernel(DownArgs a) {
  using T = FmtOf<F>;
  __shared__ DecodePlan plan;
  __shared__ float part[kDownParts][16];
  for (int i = threadIdx.x; i < (int)(sizeof(DecodePlan) / 16); i += kDownWaves * kWave)
    reinterpret_cast<uint4*>(&plan)[i] = reinterpret_cast<const uint4*>(a.plan)[i];
  __syncthreads();
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, n = min(n0 + (lane & 15), a.H - 1);
  const int active = __builtin_amdgcn_readfirstlane(plan.active);
  // Shares of K: about four jobs a wave, at least one unit each.  shares * valid <= kDownParts: an active
  // expert has up to 16 of the valid rows, so while active < 16 it is at most 16 * (32 + active - 1), up to
  // 31 two shares of 256 rows, then one.
  const int row_bytes = a.I / T::kVal * 16;
  const int shares = active ? min((4 * kDownWaves + active - 1) / active, (row_bytes + 127) >> 7) : 1;
  const int units = active * shares;
  stream<F, 1, kDepthDown<F>>(
      units > wave ? (units - wave + kDownWaves - 1) / kDownWaves : 0,
      [&](int job, auto& p, int& first, int& stride) {
        const int unit = wave + job * kDownWaves, at = unit / shares;
        const int e = __builtin_amdgcn_readfirstlane(plan.expert[at]), count = plan.count[at];
        set_rows(p, a.w, a.s, {(long long)e * a.H}, n0, n, a.I);
        p.x = reinterpret_cast<const uint8_t*>(a.h);
        p.x_off = (uint32_t)plan.rows[at][min(lane & 15, count - 1)] * (uint32_t)a.I * 2 + p.x_lane(p.g);
        first = unit - at * shares;
        stride = shares;
      },
      [&](int job) {
        const int unit = wave + job * kDownWaves;
        return Products<F, 1, 1>::steps(row_bytes, unit - unit / shares * shares, shares);
      },
      [&](int job, const f32x4 (&acc)[1]) {
        const int unit = wave + job * kDownWaves, at = unit / shares, share = unit - at * shares;
        const int count = plan.count[at];
        float scale = 1.0f;
        if (F == kInt8) scale = reinterpret_cast<const float*>(a.s)[(long long)plan.expert[at] * a.H + n];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 4 * (lane >> 4) + r;
          if (j < count) part[share * a.valid + plan.rows[at][j]][lane & 15] = F == kInt8 ? acc[0][r] * scale : acc[0][r];
        }
      });
  __syncthreads();
  const int t = threadIdx.x >> 4, c = n0 + (threadIdx.x & 15);
  if (t >= a.T || c >= a.H) return;
  float v = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int r = t * a.k + j;
    if (r >= a.valid) break;   // rows from `valid` on are not routed
    float y = 0.0f;
    for (int i = 0; i < shares; ++i) y += part[i * a.valid + r][threadIdx.x & 15];
    v = fmaf(plan.weight[r], y, v);
  }
  const long long o = (long long)t * a.H + c;
  if (a.out_bf16)
    static_cast<uint16_t*>(a.out)[o] = f32_to_bf16_bits(v);
  else
    static_cast<float*>(a.out)[o] = v;
}

template <int F, int EPL>
hipError_t launch_up(const UpArgs& a, hipStream_t stream) {
  // what fits on 256 CUs at once
  const long long items = (long long)std::min(a.valid, a.E) * a.blocks;
  const int grid = (int)std::max(1ll, std::min<long long>(items, 256 * kUpGroups<F>));
  hipLaunchKernelGGL((decode_up_kernel<F, EPL>), dim3(grid), dim3(kUpWaves * kWave), 0, stream, a);
  return hipGetLastError();
}

template <int F>
hipError_t launch_both(const UpArgs& u, const DownArgs& d, hipStream_t stream) {
  hipError_t e;
  switch ((u.E + kWave - 1) / kWave) {
    case 1: e = launch_up<F, 1>(u, stream); break;
    case 2: e = launch_up<F, 2>(u, stream); break;
    case 3: case 4: e = launch_up<F, 4>(u, stream); break;
    default: e = launch_up<F, 16>(u, stream); break;
  }
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(decode_down_kernel<F>, dim3((d.H + 15) / 16), dim3(kDownWaves * kWave), 0, stream, d);
  return hipGetLastError();
}

}  // namespace

size_t decode_plan_bytes() { return sizeof(DecodePlan); }

hipError_t launch_decode(const DecodeLaunch& q, hipStream_t stream) {
  UpArgs u{};
  u.x = static_cast<const uint8_t*>(q.x);
  u.logits = q.logits;
  u.w = static_cast<const uint8_t*>(q.w13);
  u.s = static_cast<const uint8_t*>(q.w13_scales);
  u.T = q.T;
  u.H = q.H;
  u.I = q.I;
  u.E = q.E;
  u.k = q.k;
  u.valid = q.valid;
  u.renorm = q.renorm;
  u.blocks = (q.I + 15) / 16;
  u.plan = static_cast<DecodePlan*>(q.plan);
  u.h = static_cast<uint16_t*>(q.h);
  DownArgs d{};
  d.plan = u.plan;
  d.h = u.h;
  d.w = static_cast<const uint8_t*>(q.w2);
  d.s = static_cast<const uint8_t*>(q.w2_scales);
  d.T = q.T;
  d.H = q.H;
  d.I = q.I;
  d.k = q.k;
  d.valid = q.valid;
  d.out = q.out;
  d.out_bf16 = q.out_bf16;
  switch (q.format) {
    case 0: return launch_both<kBf16>(u, d, stream);
    case 1: return launch_both<kE4m3>(u, d, stream);
    case 2: return launch_both<kInt8>(u, d, stream);
    case 3:
      if (q.group == 32) return launch_both<kInt4x32>(u, d, stream);
      if (q.group == 64) return launch_both<kInt4x64>(u, d, stream);
      return launch_both<kInt4x128>(u, d, stream);
    case 4: return launch_both<kMxfp4>(u, d, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
