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
// The bytes of the routed experts' weights bound it; they are read in whole cache lines of 8 rows a load.
// One v_mfma_f32_16x16x32_bf16 has 8 rows of each of two experts and up to 8 tokens of each: of its 16 x 16
// results the two 8 x 8 blocks where expert and token belong together are used.  So a wave works on 8 columns at
// a time, which splits the columns of small layers over more workgroups.  An expert of up to 8 tokens is listed and
// its weights are loaded once; one of more is listed twice, in general in two pairs, whose waves each load its weights.
// With an odd number of entries the last one is both halves of its pair (the same wave loads the same lines twice).
//
// The routing is recomputed by each workgroup of the first kernel (a wave a token at a time; a third launch or
// a wait between workgroups would cost more) and left for the second one.  In the first kernel 1, 2, 4 or 8 waves share
// K of 8 columns of two experts; in the second 8 or 16 waves share all experts' K of 8 output columns, so
// that a token's sum over its experts ends in one place and needs no atomics: sums are joined through LDS in a
// fixed order.
//
// First and second kernel, and the bytes of the weights that they read: bf16, 1 token, 4 experts of 2880 x 2880: 24.5
// and 15.5 us, 133 and 66 MB (5.4 and 4.3 TB/s); e4m3, 8 tokens, 30 experts of 7168 x 2048: 140 and 94 us, 870 and
// 435 MB (6.2 and 4.6); mxfp4, 4 tokens, 15 experts of 2880 x 2880: 37.5 and 25.5 us, 129 and 65 MB (3.4 and 2.5:
// rows of 1440 bytes, so that each 128 bytes are parts of two cache lines; with activations, scales and products
// left out 33 and 18 us); int4 with groups of 32, 16 tokens, 71 experts of 2048 x 768: 41.5 and 21 us, 140 and 70 MB
// (3.4 and 3.3; 8 and 3 steps a row).

#include <algorithm>
#include <type_traits>

#include "decode_plan.h"
#include "fourbit_device.h"
#include "launch.h"

namespace moe {

namespace {

enum Fmt { kBf16, kInt8, kE4m3, kInt4x32, kInt4x64, kInt4x128, kMxfp4 };

template <int F>
struct FmtOf {
  static constexpr bool kInt4 = F == kInt4x32 || F == kInt4x64 || F == kInt4x128;
  static constexpr bool kFour = kInt4 || F == kMxfp4;
  static constexpr int kBits = F == kBf16 ? 16 : kFour ? 4 : 8;
  static constexpr int kVal = 128 / kBits;            // weights in 16 bytes
  static constexpr int kX = kVal / 8;                 // MFMAs of a 64-byte piece
  static constexpr int kXBytes = kVal * 2;            // activations of 16 bytes of weights
  static constexpr int kGroup = F == kInt4x32 || F == kMxfp4 ? 32 : F == kInt4x64 ? 64 : 128;
  static constexpr int kGroups = kInt4 ? 128 / kGroup : 1;   // int4 scales of a piece
  static constexpr int kScale = kInt4 ? 4 * kGroups : F == kBf16 || F == kInt8 ? 0 : 4;   // bytes that a lane loads
  static constexpr int kXRow = 8 * kXBytes;           // bytes of a token's activations in a step
  static constexpr int kXTokens = 512 / kXRow;        // tokens of each of two experts that a load of 1 KB holds
};

// bytes of a weight row in a step: a cache line, two pieces of four lanes' 16 bytes
constexpr int kStep = 128;

// One step's weights, scales and activations of a lane.  NX: loads of activations, which hold kXTokens * NX tokens of each
// expert; NX = 8 (4 bits only): four of each 64-byte piece's channels, which go through LDS one piece after the other.
template <int F, int NM, int NX>
struct Step {
  using T = FmtOf<F>;
  uint4 w[NM][2];
  uint4 x[NX];
  uint32_t s[T::kGroups];   // bits of int4's f32 scales or e4m3's block scale, or mxfp4's four bytes
  int left;                 // uniform: bytes of the row from the step on
};

// A buffer load's offset that is past the end of any buffer here: the lane gets zeros and no memory is read.
constexpr uint32_t kPast = 0x80000000u;

__device__ __forceinline__ auto buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

template <int AUX = 0>   // 2: nontemporal
__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t rows, uint32_t lane_offset, int offset) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rows, (int)lane_offset, offset, AUX));
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

// Eight weight rows of each of two experts (NM times) times up to eight tokens of each, over a wave's steps of 128 bytes
// of the rows: first, first + stride, ...
//
// MFMA layout: the lane's weight row, of the first expert for c = lane % 16 < 8, else of the second, is column c of the
// result, the lane's token row (of the same expert) row c of the activations; g = lane / 16 picks the lane's 16 bytes
// of a 64-byte piece.  acc[m][r] becomes the sum of token row 4 g + r and weight row c, one of an expert and its own token
// where g / 2 = c / 8.
//
// Loads take whole cache lines in the lanes' order: 8 lanes a weight row's 128 bytes, one load for each expert's rows;
// activations of as many tokens as the largest expert has.  They go to the MFMA's layout through LDS of the wave.  (A
// load of weights in that layout, 16 rows for 16 lanes in a row, took the first-level cache 37 accesses where lines in
// order take 8; of activations, with every expert's eight tokens, eight loads for mxfp4's two of weights: the second
// kernel took 34 us with them and 23 without.)
//
// A lane loads the scales of one weight row, matrix and 64-byte piece, and all four lanes of a row find
// theirs in LDS (loaded by each lane for itself they took a fifth of mxfp4's time).
//
// A lane's 16 bytes are 16 or 32 channels of the narrower formats, several MFMAs' share.  Words change places between
// the lane groups (8 bits: halves, 2 swaps; 4 bits: a 4 x 4 transpose), so that each MFMA has 32
// consecutive channels and 4-bit groups have one scale in an MFMA.
//
// Addresses are a buffer's base, a scalar offset that walks along the row and 32-bit offsets of the lane that stay.
template <int F, int NM, int NX>
struct Products {
  using T = FmtOf<F>;
  using S = Step<F, NM, NX>;
  static constexpr bool kHalves = NX == 8;
  static constexpr int kXLoads = kHalves ? 4 : NX;                    // that LDS holds
  static constexpr int kXRow = kHalves ? T::kXRow / 2 : T::kXRow;     // bytes of a token there
  // LDS of a wave: weights, activations, scales
  static constexpr int kW = NM * 2048, kX = kXLoads * 1024, kLds = kW + kX + 64 * T::kScale;
  const uint8_t* w[NM][2];    // uniform: the two experts' first weight rows
  uint32_t w_bytes;           // of an expert's rows of a matrix, below kPast
  uint32_t w_off;             // the loads' row and byte
  const uint8_t* x;           // uniform
  uint32_t x_bytes;           // below kPast
  uint32_t x_off[kXLoads];    // the loads' rows and bytes; kPast where an expert has no such token
  const uint8_t* s;           // the scales that the lane loads: of its row, matrix and piece
  int row_bytes;              // of a weight row

  // byte of the lane's 8 channels of an MFMA's 32: 8 bits in the order that the swap of halves leaves
  static __device__ __forceinline__ int x_lane() {
    const int g = lane_id() >> 4;
    return T::kBits == 8 ? 32 * (g & 1) + 8 * (g & 2) : 16 * g;
  }
  // the bytes of a step that the lane loads of its weight row and of its token row
  static __device__ __forceinline__ int w_lane() { return 16 * (lane_id() & 7); }
  static __device__ __forceinline__ int x_load() { return 16 * lane_id() & (kXRow - 1); }
  // load i's token in lanes of this lane's place, and which of the two experts' it is
  static __device__ __forceinline__ int x_row(int i) { return i * (1024 / kXRow) + lane_id() / (kXRow / 16); }
  // the lane's scales: of matrix m, piece p
  static __device__ __forceinline__ int s_matrix() { return NM == 2 ? lane_id() >> 5 : 0; }
  static __device__ __forceinline__ int s_piece() { return F == kE4m3 ? 0 : (lane_id() >> 4) & 1; }

  // 4 bits: scales in a 64-byte piece
  static constexpr int kPieceGroups = 128 / T::kGroup;

  // One set of loads for every step.  Of a row's last, shorter one lanes past its end load zeros (scales: the row's
  // last ones, which end_row() brings into place), and so does each lane with `past` = kPast, past the last step of all.
  __device__ __forceinline__ void load(S& b, int at, uint32_t past) const {
    const int left = row_bytes - at;
    b.left = left;
    const int x_left = left / 16 * T::kXBytes;
    const uint32_t wo = w_off | past | (w_lane() < left ? 0u : kPast);
    const auto rows = buffer(x, x_bytes);
    const int x_at = at / 16 * T::kXBytes;
#pragma unroll
    for (int h = 0; h < NX / kXLoads; ++h) {
      const uint32_t end = past | (kXRow * h + x_load() < x_left ? 0u : kPast);
#pragma unroll
      for (int i = 0; i < kXLoads; ++i) b.x[kXLoads * h + i] = load16(rows, (x_off[i] | end) + kXRow * h, x_at);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int p = 0; p < 2; ++p)   // read once: not kept in the caches
        b.w[m][p] = load16<2>(buffer(w[m][p], w_bytes), wo, at);
    if constexpr (F == kE4m3) b.s[0] = *reinterpret_cast<const uint32_t*>(s + (at >> 7) * 4);
    if constexpr (T::kFour) {
      // the piece's first scale; rows have at least 128 channels
      const int group = min((at + 64 * s_piece()) * 2 / T::kGroup, row_bytes * 2 / T::kGroup - kPieceGroups);
      __builtin_memcpy(b.s, s + group * (F == kMxfp4 ? 1 : 4), T::kScale);
    }
  }

  // Of a row's last, shorter step: brings 4-bit scales, which were the row's last ones, into place.
  static __device__ __forceinline__ void end_row(S& b) {
    if constexpr (T::kFour) {
      // scales of the piece that the row lacks; a piece past the row has no activations left
      const int by = max(kPieceGroups - max(b.left - 64 * s_piece(), 0) * 2 / T::kGroup, 0) & (kPieceGroups - 1);
      if constexpr (F == kMxfp4) {
        b.s[0] >>= 8 * by;
      } else {
#pragma unroll
        for (int bit = 1; bit < T::kGroups; bit *= 2)
#pragma unroll
          for (int q = 0; q + bit < T::kGroups; ++q) b.s[q] = by & bit ? b.s[q + bit] : b.s[q];
      }
    }
  }

  // Loaded lines to LDS, and from there in the MFMA's layout.  16-byte chunk j of weight row r is kept at j ^ (r % 8),
  // of a token's row at j ^ (token + 8 * expert), within 128 bytes where a row has no more: neither side has bank conflicts.
  static __device__ __forceinline__ int x_chunk(int row, int chunk) {
    return kXRow * row + 16 * (chunk ^ (kXRow == 128 ? row >> 1 & 7 : (row >> 1 & 7) | (row & 1) << 3));
  }
  static __device__ __forceinline__ void put_x(uint8_t* lds, const S& b, int h) {
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      *reinterpret_cast<uint4*>(lds + kW + x_chunk(x_row(i), x_load() / 16)) = b.x[kXLoads * h + i];
  }
  static __device__ __forceinline__ void put(uint8_t* lds, const S& b) {
    const int lane = lane_id(), r = lane >> 3;
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4*>(lds + 2048 * m + 1024 * i + 128 * r + 16 * ((lane & 7) ^ r)) = b.w[m][i];
    put_x(lds, b, 0);
    if constexpr (T::kScale > 0) {
      uint32_t* to = reinterpret_cast<uint32_t*>(lds + kW + kX + T::kScale * (4 * (lane & 15) + (lane >> 4)));
#pragma unroll
      for (int i = 0; i < T::kGroups; ++i) to[i] = b.s[i];
    }
  }
  static __device__ __forceinline__ void get_weights(const uint8_t* lds, int m, int p, uint32_t (&d)[4]) {
    const int c = lane_id() & 15, g = lane_id() >> 4;
    const uint4 v = *reinterpret_cast<const uint4*>(lds + 2048 * m + 128 * c + 16 * ((4 * p + g) ^ (c & 7)));
    d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
  }
  // the activations of the step's MFMA i (of those in LDS); tokens past the loaded ones repeat the last
  static __device__ __forceinline__ bf16x8 get_x(const uint8_t* lds, int i) {
    const int c = lane_id() & 15, row = 2 * min(c & 7, kXLoads * (512 / kXRow) - 1) + (c >> 3);
    return as_bf16x8(*reinterpret_cast<const uint4*>(lds + kW + x_chunk(row, 4 * i + x_lane() / 16)));
  }
  static __device__ __forceinline__ void get_scales(const uint8_t* lds, int m, int p, uint32_t (&d)[T::kGroups]) {
    const uint32_t* from = reinterpret_cast<const uint32_t*>(lds + kW + kX + T::kScale * (4 * (lane_id() & 15) + 2 * m + p));
#pragma unroll
    for (int i = 0; i < T::kGroups; ++i) d[i] = from[i];
  }

  // Between LDS accesses of lanes of the wave that depend on each other.  The hardware keeps a wave's in order; this holds
  // the compiler to it, which sees the accesses of one lane only.  No instruction.
  static __device__ __forceinline__ void keep_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

  static __device__ __forceinline__ void use(uint8_t* lds, const S& b, f32x4 (&acc)[NM]) {
    f32x4 part[NM];   // e4m3: the block's sum
#pragma unroll
    for (int m = 0; m < NM; ++m) part[m] = f32x4{0, 0, 0, 0};
    keep_order();
    put(lds, b);
    keep_order();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (T::kFour) __builtin_amdgcn_sched_barrier(0);   // one piece's operands at a time
      if (kHalves && p == 1) {   // behind the first piece's reads
        keep_order();
        put_x(lds, b, 1);
        keep_order();
      }
      uint32_t d[NM][4], s[NM][T::kGroups];
#pragma unroll
      for (int m = 0; m < NM; ++m) get_weights(lds, m, p, d[m]);
      bf16x8 x[T::kX];
#pragma unroll
      for (int q = 0; q < T::kX; ++q) x[q] = get_x(lds, kHalves ? q : T::kX * p + q);
      if constexpr (T::kFour) {
#pragma unroll
        for (int m = 0; m < NM; ++m) get_scales(lds, m, p, s[m]);
      }
      if constexpr (F == kBf16) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              x[0], as_bf16x8(make_uint4(d[m][0], d[m][1], d[m][2], d[m][3])), acc[m], 0, 0, 0);
      } else if constexpr (F == kInt8 || F == kE4m3) {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          // rows 2, 3 of the first half change places with rows 0, 1 of the second
          const auto lo = __builtin_amdgcn_permlane32_swap(d[m][0], d[m][2], false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(d[m][1], d[m][3], false, false);
          f32x4& sum = F == kE4m3 ? part[m] : acc[m];
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[0], unpack8<F>(lo[0], hi[0]), sum, 0, 0, 0);
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[1], unpack8<F>(lo[1], hi[1]), sum, 0, 0, 0);
        }
      } else if constexpr (F == kMxfp4) {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          transpose4(d[m]);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                x[q], as_bf16x8(unpack_mxfp4(d[m][q], s[m][0] >> (8 * q) & 0xffu)), acc[m], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int m = 0; m < NM; ++m) transpose4(d[m]);
        // a group's sum of code * x starts from -8 * sum of x
        const bf16x8 minus8 = as_bf16x8(make_uint4(0xc100c100u, 0xc100c100u, 0xc100c100u, 0xc100c100u));
        constexpr int kPer = 4 / T::kGroups;   // MFMAs of a scale
#pragma unroll
        for (int q0 = 0; q0 < 4; q0 += kPer) {
          f32x4 group[NM];
#pragma unroll
          for (int q = q0; q < q0 + kPer; ++q) {
            const f32x4 start = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[q], minus8, f32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
            for (int m = 0; m < NM; ++m) {
              const f32x4 one = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  x[q], as_bf16x8(unpack_int4_ordered(d[m][q])), start, 0, 0, 0);
#pragma unroll
              for (int r = 0; r < 4; ++r) group[m][r] = q == q0 ? one[r] : group[m][r] + one[r];
            }
          }
#pragma unroll
          for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[m][r] = fmaf(group[m][r], __uint_as_float(s[m][q0 / kPer]), acc[m][r]);
          // here and now: moved behind the branches that follow, the step's 16 products stay in registers until then
#pragma unroll
          for (int m = 0; m < NM; ++m) asm volatile("" : "+v"(acc[m]));
        }
      }
    }
    if constexpr (F == kE4m3) {
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        uint32_t s[1];
        get_scales(lds, m, 0, s);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[m][r] = fmaf(part[m][r], __uint_as_float(s[0]), acc[m][r]);
      }
    }
  }

  // steps of a share of a row
  static __device__ __forceinline__ int steps(int row_bytes, int first, int stride) {
    const int units = (row_bytes + kStep - 1) / kStep;
    return first < units ? (units - first + stride - 1) / stride : 0;
  }
};

// Streams the products of jobs 0 to jobs - 1 through a wave: a step's loads are in flight during the MFMAs
// of the step before, across the ends of jobs.  (With 16 waves on a CU two or three steps ahead are no
// faster: bf16's first kernel 25.4 us for 24.9, mxfp4's second 27.1 for 25.4, e4m3's 93 for 91.)
//
// share(job, first, stride): the job's share of K, at least one step; start(job, products) sets its streams;
// finish(job, sums) takes its sums.
//
// Every step loads, past the last one zeros that cost no memory access, so that the compiler's count of loads in
// flight holds on every path.
template <int F, int NM, int NX, typename Share, typename Start, typename Finish>
__device__ __forceinline__ void stream(uint8_t* lds, int jobs, int row_bytes, Share&& share, Start&& start,
                                       Finish&& finish) {
  using P = Products<F, NM, NX>;
  if (jobs <= 0) return;
  struct Cursor {   // a step of a job
    int job, step, n, first, stride;
    __device__ __forceinline__ int at() const { return (first + step * stride) * kStep; }
  };
  auto begin = [&](Cursor& c, int job) {
    c.job = job;
    c.step = 0;
    share(job, c.first, c.stride);
    c.n = P::steps(row_bytes, c.first, c.stride);
  };
  P p;
  p.row_bytes = row_bytes;
  Cursor get, now;
  begin(get, 0);
  begin(now, 0);
  start(0, p);
  uint32_t past = 0;
  auto load = [&](Step<F, NM, NX>& b) {
    p.load(b, get.at(), past);
    if (get.step + 1 < get.n) {
      ++get.step;
    } else if (get.job + 1 < jobs) {
      begin(get, get.job + 1);
      start(get.job, p);
    } else {
      past = kPast;
    }
  };
  Step<F, NM, NX> b;
  load(b);
  f32x4 acc[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) acc[m] = f32x4{0, 0, 0, 0};
  while (true) {
    if (b.left < kStep) P::end_row(b);
    P::use(lds, b, acc);
    // the loads stay behind the products of the step whose registers they take: hoisted, they need others
    __builtin_amdgcn_sched_barrier(0);
    load(b);
    __builtin_amdgcn_sched_barrier(0);
    if (++now.step < now.n) continue;
    finish(now.job, acc);
    if (now.job + 1 == jobs) return;
    begin(now, now.job + 1);
#pragma unroll
    for (int m = 0; m < NM; ++m) acc[m] = f32x4{0, 0, 0, 0};
  }
}

// Calls f with the loads of activations that hold the tokens of the largest listed expert.
template <int F, typename Fn>
__device__ __forceinline__ void with_x_loads(int most, Fn&& f) {
  constexpr int kBits = FmtOf<F>::kBits;
  const int n = (most + FmtOf<F>::kXTokens - 1) / FmtOf<F>::kXTokens;
  if (n <= 1) return f(std::integral_constant<int, 1>{});
  if constexpr (kBits == 16) {
    f(std::integral_constant<int, 2>{});
  } else {
    if (n <= 2) return f(std::integral_constant<int, 2>{});
    if constexpr (kBits == 8) {
      f(std::integral_constant<int, 4>{});
    } else {
      if (n <= 4) return f(std::integral_constant<int, 4>{});
      f(std::integral_constant<int, 8>{});
    }
  }
}
template <int F>
constexpr int kMostXLds = FmtOf<F>::kBits == 16 ? 2 : 4;   // loads that go through LDS
template <int F, int NM>
constexpr int kWaveLds = Products<F, NM, kMostXLds<F>>::kLds;

constexpr int kWaves = 8;
constexpr int kUpGroups = 512;     // workgroups of the first kernel: two on each of 256 CUs
template <int W>
constexpr int kDownParts = 64 * W;    // routed rows times shares of K that the second kernel's LDS holds

struct UpArgs {
  const uint8_t* x;       // [T, H] bf16
  const float* logits;    // [T, E]
  const uint8_t* w;       // [E, 2I, H]
  const uint8_t* s;
  int T, H, I, E, k, valid, renorm;
  int blocks;             // ceil(I / 8)
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

// The streams of a wave on columns n0 to n0 + 7 of the listed experts `at` and `at` + 1 (past the list's end: of the
// last one again).  Expert e's NM blocks of N weight rows of K channels begin at row e * NM * N; columns past N repeat
// the last one.  N rows are below 2 GiB, and so are the activations, x_rows rows of K at x, of which `rows` has the tokens'.
template <int F, int NM, int NX>
__device__ __forceinline__ void set_rows(Products<F, NM, NX>& p, const DecodePlan& plan, int at, int n0, const uint8_t* w,
                                         const uint8_t* s, int N, int K, const void* x, int x_rows,
                                         const uint8_t (&rows)[kDecodeRows][8]) {
  using P = Products<F, NM, NX>;
  const int sb = scale_bytes<F>(K);
  const int e[2] = {__builtin_amdgcn_readfirstlane(plan.expert[at]),
                    __builtin_amdgcn_readfirstlane(plan.expert[min(at + 1, plan.entries - 1)])};
  p.w_bytes = (uint32_t)N * (uint32_t)p.row_bytes;
  p.w_off = (uint32_t)min(n0 + (lane_id() >> 3), N - 1) * (uint32_t)p.row_bytes + P::w_lane();
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) p.w[m][i] = w + ((long long)e[i] * NM + m) * N * p.row_bytes;
  const int c = lane_id() & 15;
  const long long row = ((long long)(c < 8 ? e[0] : e[1]) * NM + P::s_matrix()) * N + min(n0 + (c & 7), N - 1);
  p.s = s + (F == kE4m3 ? row >> 7 : row) * sb;
  p.x = static_cast<const uint8_t*>(x);
  p.x_bytes = (uint32_t)(x_rows * K) * 2;
  auto row_of = [&](int half, int token, int byte) {
    const int entry = at + half;
    return entry < plan.entries && token < plan.count[entry] ? (uint32_t)rows[entry][token] * (uint32_t)K * 2 + byte : kPast;
  };
#pragma unroll
  for (int i = 0; i < P::kXLoads; ++i) p.x_off[i] = row_of(P::x_row(i) & 1, P::x_row(i) >> 1, P::x_load());
}

// Top-k routing of one token by a wave, with the ids and weights of route_device.h's route_token: k rounds of a
// maximum over the lanes.  Logits are compared as integers that order as they do, so that a step of
// the maximum is one instruction; the lowest id of equal ones is the first lane that has the maximum, of the first
// 64 experts that have it.  (Every workgroup routes every token: 16 of 128 experts, 8 each, were half of the first kernel's
// instructions with route_token.)
//
// EPL: experts of a lane.  The rounds are a part of the first kernel that nothing hides: with 4 for 128 experts, 16
// tokens and 8 each, it took 44.8 us for 41.6 with 2.
template <int EPL>
__device__ __forceinline__ void route(const UpArgs& a, int t, int* ids, float* weights) {
  const int lane = lane_id();
  const float* row = a.logits + (size_t)t * a.E;
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + kWave * i;
    const uint32_t b = __float_as_uint((e < a.E ? row[e] : 0.0f) + 0.0f);   // -0 becomes 0
    key[i] = e < a.E ? max(b ^ ((uint32_t)((int)b >> 31) | 0x80000000u), 1u) : 0u;   // 0: not there, or taken
  }
  auto value = [](uint32_t u) { return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); };
  uint32_t all[EPL];   // the softmax over all logits needs them again
#pragma unroll
  for (int i = 0; i < EPL; ++i) all[i] = key[i];
  uint32_t my_key = 0, top = 0;
  int my_id = 0;
  for (int j = 0; j < a.k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = max(m, key[i]);
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, m, 0x128, 0xf, 0xf, false));   // row_ror by 8, 4, 2, 1
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, m, 0x124, 0xf, 0xf, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, m, 0x122, 0xf, 0xf, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, m, 0x121, 0xf, 0xf, false));
    const uint32_t best = max(max((uint32_t)__builtin_amdgcn_readlane(m, 0), (uint32_t)__builtin_amdgcn_readlane(m, 16)),
                              max((uint32_t)__builtin_amdgcn_readlane(m, 32), (uint32_t)__builtin_amdgcn_readlane(m, 48)));
    bool found = false;
    int id = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint64_t who = __ballot(key[i] == best);
      const bool here = !found && who != 0;
      const int l = __builtin_ctzll(who | (1ull << 63));
      id = here ? kWave * i + l : id;
      key[i] = here && lane == l ? 0u : key[i];
      found |= here;
    }
    if (j == 0) top = best;
    if (lane == j) {
      my_key = best;
      my_id = id;
    }
  }
  const float ex = lane < a.k ? expf(value(my_key) - value(top)) : 0.0f;
  float denom;
  if (a.renorm) {
    denom = wave_sum(ex);
  } else {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + kWave * i < a.E) s += expf(value(all[i]) - value(top));
    denom = wave_sum(s);
  }
  if (lane < a.k) {
    const int r = t * a.k + lane;
    ids[r] = r < a.valid ? my_id : a.E;
    weights[r] = r < a.valid ? ex / denom : 0.0f;
  }
}

// Routes the tokens and lists the experts that have rows, in the order of their first (and their ninth) row, with their
// rows in ascending order.
template <int EPL>
__device__ __forceinline__ void make_plan(const UpArgs& a, DecodePlan& plan, uint32_t* tokens, uint16_t (*index)[2],
                                          int* ids) {
  const int wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < a.E; e += kWaves * kWave) tokens[e] = 0;
  if (threadIdx.x == 0) plan.most = 1;
  for (int t = wave; t < a.T; t += kWaves) route<EPL>(a, t, ids, plan.weight);
  __syncthreads();
  const int r = threadIdx.x;   // T k <= 256
  const int e = r < a.T * a.k ? ids[r] : a.E;
  const int t = r / a.k;
  const bool live = (unsigned)e < (unsigned)a.E;
  if (live) atomicOr(&tokens[e], 1u << t);
  __syncthreads();
  const uint32_t mine = live ? tokens[e] : 0;
  const int rank = __popc(mine & ((1u << t) - 1));
  const bool first = live && (rank & 7) == 0;
  // position among the first rows of entries: this wave's by ballot, the waves' by LDS
  const uint64_t firsts = __ballot(first);
  if (lane_id() == 0) ids[kDecodeRows + wave] = __popcll(firsts);
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const int n = ids[kDecodeRows + i];
    before += i < wave ? n : 0;
    all += n;
  }
  if (first) {
    const int at = before + __popcll(firsts & ((1ull << lane_id()) - 1));
    index[e][rank >> 3] = (uint16_t)at;
    plan.expert[at] = (uint16_t)e;
    plan.count[at] = (uint8_t)min(__popc(mine) - rank, 8);
    atomicMax(&plan.most, min(__popc(mine), 8));
  }
  if (threadIdx.x == 0) plan.entries = all;
  __syncthreads();
  if (live) {
    const int at = index[e][rank >> 3];
    plan.id[r] = (uint16_t)e;
    plan.rows[at][rank & 7] = (uint8_t)r;
    plan.tokens[at][rank & 7] = (uint8_t)t;
  }
  __syncthreads();
}

template <int F, int EPL>
__global__ __launch_bounds__(kWaves * kWave, 4) void decode_up_kernel(UpArgs a) {
  using T = FmtOf<F>;
  __shared__ DecodePlan plan;
  // The waves' LDS.  Before the streams the lists of make_plan(), at an item's end its sums.
  struct Lists {
    uint32_t tokens[EPL * kWave];
    uint16_t index[EPL * kWave][2];
    int ids[kDecodeRows + kWaves];
  };
  __shared__ union {
    Lists lists;
    __attribute__((aligned(16))) uint8_t lines[kWaves][kWaveLds<F, 2>];
  } lds;
  static_assert(sizeof(lds) + sizeof(DecodePlan) <= 80 << 10, "two workgroups on a CU");
  make_plan<EPL>(a, plan, lds.lists.tokens, lds.lists.index, lds.lists.ids);
  if (blockIdx.x == 0) {   // for the second kernel
    const uint4* from = reinterpret_cast<const uint4*>(&plan);
    for (int i = threadIdx.x; i < (int)(sizeof(DecodePlan) / 16); i += kWaves * kWave)
      reinterpret_cast<uint4*>(a.plan)[i] = from[i];
  }
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int entries = __builtin_amdgcn_readfirstlane(plan.entries);
  const int items = (entries + 1) / 2 * a.blocks;   // (two experts, 8 columns)
  const int units = (a.H / T::kVal * 16 + kStep - 1) / kStep;
  // Waves that share an item's K: more while each has three steps or where waves are left over
  int split = 1;
  while (split < kWaves && 2 * split <= units &&
         (units >= 6 * split || 2 * split * items <= (int)gridDim.x * kWaves))
    split *= 2;
  const int share = wave % split, group = wave / split;
  const int groups = (int)gridDim.x * (kWaves / split);
  const int rounds = (items + groups - 1) / groups;
  const int my_first = (int)blockIdx.x * (kWaves / split) + group;
  const int jobs = items > my_first ? (items - my_first + groups - 1) / groups : 0;   // rounds or one less
  auto item_of = [&](int job, int& at, int& n0) {
    const int item = my_first + job * groups, pair = item / a.blocks;
    at = 2 * pair;
    n0 = (item - pair * a.blocks) * 8;
  };
  auto store = [&](int at, int half, int token, int col, float gate, float up) {
    if (at + half < entries && token < plan.count[at + half] && col < a.I) {
      if (F == kInt8) {
        const float* s = reinterpret_cast<const float*>(a.s) + (long long)plan.expert[at + half] * 2 * a.I + col;
        gate *= s[0];
        up *= s[a.I];
      }
      a.h[(long long)plan.rows[at + half][token] * a.I + col] = f32_to_bf16_bits(silu_mul(gate, up));
    }
  };
  const int half = (lane >> 3) & 1, token0 = 4 * ((lane >> 4) & 1);
  const bool mine = lane >> 5 == half;   // the lane's sums are of a token and its own expert
  auto finish = [&](int job, const f32x4 (&v)[2]) {
    int at, n0;
    item_of(job, at, n0);
    if (split == 1) {
      if (mine)
#pragma unroll
        for (int r = 0; r < 4; ++r) store(at, half, token0 + r, n0 + (lane & 7), v[0][r], v[1][r]);
      return;
    }
    auto part = [&](int w) { return reinterpret_cast<float(*)[2][8][8]>(lds.lines[w]); };   // [gate or up]
    if (mine)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) part(wave)[m][half][token0 + r][lane & 7] = v[m][r];
    __syncthreads();
    const int u = share * kWave + lane;   // expert, token and column
    if (u < 128) {
      float sum[2] = {0.0f, 0.0f};
      for (int i = 0; i < split; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m) sum[m] += part(wave - share + i)[m][u >> 6][(u >> 3) & 7][u & 7];
      store(at, u >> 6, (u >> 3) & 7, n0 + (u & 7), sum[0], sum[1]);
    }
    __syncthreads();
  };
  with_x_loads<F>(__builtin_amdgcn_readfirstlane(plan.most), [&](auto nx) {
    constexpr int NX = decltype(nx)::value;
    stream<F, 2, NX>(
        lds.lines[wave], jobs, a.H / T::kVal * 16,
        [&](int, int& first, int& stride) {
          first = share;
          stride = split;
        },
        [&](int job, auto& p) {
          int at, n0;
          item_of(job, at, n0);
          set_rows(p, plan, at, n0, a.w, a.s, a.I, a.H, a.x, a.T, plan.tokens);
        },
        finish);
  });
  if (split > 1 && jobs < rounds) {   // the other groups' last item
    __syncthreads();
    __syncthreads();
  }
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

template <int F, int W>   // W: waves of a workgroup
__global__ __launch_bounds__(W * kWave, 4) void decode_down_kernel(DownArgs a) {
  using T = FmtOf<F>;
  __shared__ DecodePlan plan;
  __shared__ float part[kDownParts<W>][8];
  __shared__ __attribute__((aligned(16))) uint8_t lines[W][kWaveLds<F, 1>];
  static_assert(sizeof(plan) + sizeof(part) + sizeof(lines) <= (80 << 10) * (W / kWaves), "16 waves on a CU");
  for (int i = threadIdx.x; i < (int)(sizeof(DecodePlan) / 16); i += W * kWave)
    reinterpret_cast<uint4*>(&plan)[i] = reinterpret_cast<const uint4*>(a.plan)[i];
  __syncthreads();
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 8;
  const int entries = __builtin_amdgcn_readfirstlane(plan.entries), pairs = (entries + 1) / 2;
  // Shares of K: about four jobs a wave, at least one unit each.  shares * valid <= 64 W: a pair
  // has up to 16 of the valid rows, all of them at most 256.
  const int units = (a.I / T::kVal * 16 + kStep - 1) / kStep;
  const int shares = pairs ? max(min(4 * W / pairs, units), 1) : 1;
  const int all = pairs * shares;
  with_x_loads<F>(__builtin_amdgcn_readfirstlane(plan.most), [&](auto nx) {
    constexpr int NX = decltype(nx)::value;
    stream<F, 1, NX>(
        lines[wave], all > wave ? (all - wave + W - 1) / W : 0, a.I / T::kVal * 16,
        [&](int job, int& first, int& stride) {
          const int unit = wave + job * W;
          first = unit - unit / shares * shares;
          stride = shares;
        },
        [&](int job, auto& p) {
          const int at = 2 * ((wave + job * W) / shares);
          set_rows(p, plan, at, n0, a.w, a.s, a.H, a.I, a.h, a.T * a.k, plan.rows);
        },
        [&](int job, const f32x4 (&acc)[1]) {
          const int unit = wave + job * W, pair = unit / shares, share = unit - pair * shares;
          const int half = (lane >> 3) & 1, token0 = 4 * ((lane >> 4) & 1), at = 2 * pair + half;
          if (lane >> 5 != half || at >= entries) return;
          const int count = plan.count[at];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (token0 + r < count) part[share * a.valid + plan.rows[at][token0 + r]][lane & 7] = acc[0][r];
        });
  });
  __syncthreads();
  const int t = threadIdx.x >> 3, c = n0 + (threadIdx.x & 7);
  if (t >= a.T || c >= a.H) return;
  float v = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int r = t * a.k + j;
    if (r >= a.valid) break;   // rows from `valid` on are not routed
    float y = 0.0f;
    for (int i = 0; i < shares; ++i) y += part[i * a.valid + r][threadIdx.x & 7];
    if (F == kInt8) y *= reinterpret_cast<const float*>(a.s)[(long long)plan.id[r] * a.H + c];
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
  // an expert is listed once for eight of its rows
  const long long items = ((long long)std::min(a.valid, a.E + a.valid / 8) + 1) / 2 * a.blocks;
  const int grid = (int)std::max(1ll, std::min<long long>(items, kUpGroups));
  hipLaunchKernelGGL((decode_up_kernel<F, EPL>), dim3(grid), dim3(kWaves * kWave), 0, stream, a);
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
  // Up to one workgroup a CU they have 16 waves, else 8, two on a CU.  The layer with 8 and with 16, in us: H 1024, I 2048,
  // 4 of 32 experts, 16 tokens, bf16 85.6 and 68.9, int4 46.5 and 42.7; H 2048, I 5632, 2 of 8, 4 tokens, bf16 70.6 and 63.6,
  // int8 47.8 and 42.9; H = I = 1440, 4 of 32, 16 tokens, 8 of them with one expert, int4 54.3 and 53.1, int8 65.5 and 60.1.  Over
  // H from 512 to 2048, 1 to 16 tokens and all formats 16 lose at most 4% (one token in bf16, 20.1 and 20.9), and up
  // to 2% in 4 bits where experts have up to four tokens (H 1024, I 1440, 4 of 32, 16 tokens, mxfp4 37.7 and 38.6).
  const int blocks = (d.H + 7) / 8;
  if (blocks <= kUpGroups / 2)
    hipLaunchKernelGGL((decode_down_kernel<F, 2 * kWaves>), dim3(blocks), dim3(2 * kWaves * kWave), 0, stream, d);
  else
    hipLaunchKernelGGL((decode_down_kernel<F, kWaves>), dim3(blocks), dim3(kWaves * kWave), 0, stream, d);
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
  u.blocks = (q.I + 7) / 8;
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
