// fourbit.hip -- grouped products with 4-bit weights and group scales, for few rows per expert:
//
//   C[p, n] = sum_k A[row(p), k] * W[e(p), n, k]         (optionally silu(gate) * up)
//
// int4: W = (code - 8) * scale, f32 scales per 32, 64 or 128 channels.  mxfp4: W = e2m1(code) *
// 2^(scale - 127), one e8m0 byte per 32 channels.  Codes are [E, N, K/2], the even channel in the
// low nibble.
//
// The bytes of the weights of the experts that have rows bound it: they are read once per 16 rows.
// The sixteen rows of v_mfma_f32_16x16x32_bf16 make the products of 1 to 16 rows cost the same.
// Two kernels: fourbit_stream_kernel where eight waves can hold the activations of a whole row in
// registers (K to 7168, int4 groups of 32 to 5120), fourbit_kernel for longer rows.
//
// mxfp4: e2m1 * 2^s is exact in bf16 (while normal), so the scale is applied while unpacking
// (v_cvt_scalef32_pk_bf16_fp4).
// int4: code * scale is not exact in bf16, so the MFMA runs on the codes 0 to 15 and the scale
// multiplies its f32 result; MFMAs have 32 consecutive channels, all of one scale, after a 4 x 4
// transpose of words between the lane groups (v_permlane32_swap, v_permlane16_swap).  The offset
// leaves as -8 * sum_g scale_g * (sum of the group's activations): in the streaming kernel one
// 16x16x4 f32 product per four groups of sums that are kept with the activations, next to those
// groups' own products, in the other a second MFMA with the constant weight -8.  The rounded sums
// have at most (15 + 8) |a| per channel where the true terms have up to 8 |a|.

#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "direct_load.h"
#include "launch.h"
#include "moe.h"
#include "rows_device.h"

namespace moe {

typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4;
typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;

__device__ __forceinline__ bf16x8 as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8, v); }

// 4 x 4 transpose of words between the four 16-lane rows of a wave: word j of row q becomes
// word q of row j
__device__ __forceinline__ void transpose4(uint32_t (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // upper half of r[i] with lower half of r[i + 2]
    const auto s = __builtin_amdgcn_permlane32_swap(r[i], r[i + 2], false, false);
    r[i] = s[0];
    r[i + 2] = s[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {   // odd rows of r[i] with even rows of r[i + 1]
    const auto s = __builtin_amdgcn_permlane16_swap(r[i], r[i + 1], false, false);
    r[i] = s[0];
    r[i + 1] = s[1];
  }
}

// eight int4 codes -> bf16 0 to 15, in the channel order 0 2 4 6 1 3 5 7: as an e4m3 byte a code
// is code * 2^-9 (subnormal below 8, and the first binade goes on in the same steps)
__device__ __forceinline__ uint4 unpack_int4(uint32_t v) {
  const uint32_t even = v & 0x0f0f0f0fu, odd = (v >> 4) & 0x0f0f0f0fu;
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, true));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, false));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, true));
  return r;
}

// eight activations into the same order
__device__ __forceinline__ uint4 order_int4(uint4 a) {
  return make_uint4(__builtin_amdgcn_perm(a.y, a.x, 0x05040100u), __builtin_amdgcn_perm(a.w, a.z, 0x05040100u),
                    __builtin_amdgcn_perm(a.y, a.x, 0x07060302u), __builtin_amdgcn_perm(a.w, a.z, 0x07060302u));
}

// eight e2m1 codes -> bf16 code * 2^(e8m0 - 127), in channel order; the conversion takes its scale
// from an f32's exponent bits
__device__ __forceinline__ uint4 unpack_mxfp4(uint32_t v, uint32_t e8m0) {
  const float scale = __uint_as_float(e8m0 << 23);
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3));
  return r;
}

// The row blocks of a launch: every expert's rows in blocks of 16, expert by expert.  Each lane keeps
// the running count of its consecutive experts' blocks; all 64 lanes take part in each call.  Offsets
// that do not ascend have no blocks: the counts and rows below hold only where they do.
struct RowBlock {
  int e, lo, hi;   // rows [lo, hi) of expert e
};

// a value that is the same in all lanes, into a scalar register (quotients are computed in vector ones)
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

struct RowBlocks {
  const int* offsets;
  int E, M_rows, per;
  static constexpr int BM = 16;
  int lo0, hi0, mine, incl;

  __device__ __forceinline__ int at(int e) const { return min(max(offsets[min(e, E)], 0), M_rows); }
  __device__ __forceinline__ int blocks(int lo, int hi) const { return max(hi - lo + BM - 1, 0) / BM; }

  __device__ __forceinline__ RowBlocks(const int* offsets_, int E_, int M_rows_)
      : offsets(offsets_), E(E_), M_rows(M_rows_), per((E_ + kWave - 1) / kWave) {
    const int lane = lane_id();
    lo0 = at(lane * per);
    mine = 0;
    bool ascend = true;
    for (int i = 0, lo = lo0; i < per; ++i) {
      const int hi = at(lane * per + i + 1);
      ascend &= lo <= hi;
      mine += blocks(lo, hi);
      lo = hi;
      if (i == 0) hi0 = hi;
    }
    if (__ballot(ascend) != ~0ull) mine = 0;
    incl = mine;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int up = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += up;
    }
  }

  __device__ __forceinline__ int count() const { return __builtin_amdgcn_readlane(incl, 63); }

  __device__ __forceinline__ RowBlock find(int block) const {   // 0 <= block < count()
    const int owner = __builtin_ctzll(__ballot(incl > block) | (1ull << 63));
    int rest = block - (__builtin_amdgcn_readlane(incl, owner) - __builtin_amdgcn_readlane(mine, owner));
    int lo = __builtin_amdgcn_readlane(lo0, owner), hi = __builtin_amdgcn_readlane(hi0, owner);
    int i = 0;
    for (; i + 1 < per && rest >= blocks(lo, hi); ++i) {
      rest -= blocks(lo, hi);
      lo = hi;
      hi = uniform(at(owner * per + i + 2));
    }
    return {uniform(owner * per + i), uniform(lo + rest * BM), uniform(min(lo + (rest + 1) * BM, hi))};
  }
};

struct FourbitArgs {
  const uint16_t* A;
  const int* a_rows;   // null: row p of A
  int a_div;
  int A_rows;
  const uint8_t* codes;
  const void* scales;
  const int* offsets;
  int E, M_rows, N, K;
  void* C;
  bool c_f32;
};

constexpr int kFbWaves = 4;
constexpr int kStep = 256;   // channels of a step: 128 bytes of a weight row, one cache line

// Two registers of a wave, each 8 weight rows x 128 bytes (lane 16 q + c: row c % 8, 16-byte piece
// q + 4 (c / 8)), into the first and second 64 bytes of all 16 rows (lane 16 q + c: row c, piece q)
__device__ __forceinline__ void halves(uint32_t& a, uint32_t& b) {
  // lanes 8..15 of each row of 16 take the other register's lanes 0..7, and the other way round
  const uint32_t first = __builtin_amdgcn_update_dpp(a, b, 0x128, 0xf, 0xc, false);    // row_ror:8
  const uint32_t second = __builtin_amdgcn_update_dpp(b, a, 0x128, 0xf, 0x3, false);
  a = first;
  b = second;
}

// LDS of a weight row's scales: whole steps (the missing channels of the last one have scales that
// do no harm) and one step of padding, so that the 16 rows of a tile start in different banks.
template <bool kInt4, int kGroup>
constexpr int kStepScaleBytes = kStep / kGroup * (kInt4 ? 4 : 1);
__host__ __device__ constexpr int scale_row_bytes(long long K, int step_bytes) {
  return (int)((K + kStep - 1) / kStep + 1) * step_bytes;
}

// Copies the scales of a workgroup's weight rows to LDS: 16 lanes a row, 4 bytes a lane (rows of
// scales start at any byte, global loads take any address).  row(i) is the weight row of LDS row i.
template <bool kInt4, int kGroup, int kRows, typename Row>
__device__ __forceinline__ void stage_scales(const uint8_t* __restrict__ scales, Row row, int K, uint8_t* lds) {
  const int row_bytes = K / kGroup * (kInt4 ? 4 : 1);
  const int stride = scale_row_bytes(K, kStepScaleBytes<kInt4, kGroup>);
  const int used = stride - kStepScaleBytes<kInt4, kGroup>;
  for (int b = (threadIdx.x & 15) * 4; b < used; b += 64) {
#pragma unroll 4
    for (int i = threadIdx.x >> 4; i < kRows; i += kFbWaves * 4) {
      const uint8_t* src = scales + (size_t)row(i) * row_bytes + b;
      uint32_t v = kInt4 ? 0u : 0x7f7f7f7fu;   // 0, or 2^0
      if (b + 4 <= row_bytes)
        __builtin_memcpy(&v, src, 4);
      else
        for (int j = 0; b + j < row_bytes; ++j) v = (v & ~(0xffu << (8 * j))) | (uint32_t)src[j] << (8 * j);
      *reinterpret_cast<uint32_t*>(lds + i * stride + b) = v;
    }
  }
}

// Long weight rows: blocks of 16 rows of an expert, NT weight tiles of 16 rows (with SiLU * up the even
// ones are gate and the odd ones up).  kGroup: channels per scale (mxfp4: 32).  The waves split K and
// join their f32 sums in LDS in wave order.  A load instruction takes whole 128-byte lines of 8 weight
// rows, which `halves` and transpose4 bring into the MFMA's order: on rows of 2048, which stream now, lane
// loads of 64 bytes of 16 rows took 349 us where whole lines took 202 (int4 groups of 128, 128 routes over
// 256 experts of 7168 x 2048; streamed 166).  8 experts of 4096 x 14336: 64 rows on all of them (250 MB, 40 us
// at the rate of a read) take 63 us in mxfp4 and 70 in int4 groups of 128, 2 rows on two (62 MB, 10 us) 32 and
// 38: a wave has one step of its tiles in flight.
template <bool kInt4, int kGroup, bool kSilu, int NT>
__global__ __launch_bounds__(kFbWaves * 64, 4) void fourbit_kernel(FourbitArgs p) {
  constexpr int BM = 16;
  constexpr int kCols = (kSilu ? NT / 2 : NT) * 16;   // output columns
  constexpr int kScaleBytes = kInt4 ? 4 : 1;
  constexpr int kScaleWords = kStepScaleBytes<kInt4, kGroup> / 4;   // scales of a row per step
  // the scales of all tiles' rows, and after the loop the waves' sums [wave][tile][row][16]
  extern __shared__ __align__(16) uint8_t shared[];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int n_out = kSilu ? p.N / 2 : p.N;
  const int groups = (n_out + kCols - 1) / kCols;
  const int block = uniform(blockIdx.x / groups), n0 = ((int)blockIdx.x - block * groups) * kCols;
  const RowBlocks rows_of(p.offsets, p.E, p.M_rows);
  const int past = block - rows_of.count();
  RowBlock blk;
  if (past < 0) {
    blk = rows_of.find(block);
  } else {   // rows without an expert
    const int lo = (int)min((long long)rows_of.at(p.E) + (long long)past * BM, (long long)p.M_rows);
    blk = {-1, lo, (int)min((long long)lo + BM, (long long)p.M_rows)};
  }
  auto store = [&](int r, int n, float v) {
    const size_t at = (size_t)r * n_out + n;
    if (p.c_f32)
      static_cast<float*>(p.C)[at] = v;
    else
      static_cast<uint16_t*>(p.C)[at] = f32_to_bf16_bits(v);
  };
  if (blk.e < 0) {   // rows without an expert are zero
    for (int i = threadIdx.x; i < (blk.hi - blk.lo) * kCols; i += kFbWaves * 64)
      if (n0 + i % kCols < n_out) store(blk.lo + i / kCols, n0 + i % kCols, 0.0f);
    return;
  }
  const int K = p.K;
  // the expert's codes, under 2 GiB: an offset with the top bit set is past their end and loads zeros
  const auto codes = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.codes) + (size_t)blk.e * p.N * (K / 2), 0, (uint32_t)p.N * (uint32_t)(K / 2), 0x00020000);
  // weight row `i` of tile t; rows past the last repeat it
  auto wrow = [&](int t, int i) {
    return (uint32_t)((kSilu && (t & 1) ? n_out : 0) + min(n0 + (kSilu ? t / 2 : t) * 16 + i, n_out - 1));
  };
  const int piece = q + 4 * (col >> 3);   // this lane's 16 bytes of a step when it loads codes
  uint32_t wat[NT][2];                    // where it loads codes of rows col % 8 and 8 + col % 8
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int h = 0; h < 2; ++h) wat[t][h] = wrow(t, (col & 7) + 8 * h) * (uint32_t)(K / 2) + 16 * piece;
  }
  int arow = min(blk.lo + col, blk.hi - 1);   // surplus rows repeat the last
  if (p.a_rows) arow = min(max(p.a_rows[arow] / p.a_div, 0), p.A_rows - 1);
  const uint16_t* ap = p.A + (size_t)arow * K;
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  struct Weights {
    uint4 c[2];
  };
  // K % 32 == 0: a lane's 32 channels are all in the row or none
  auto load_weights = [&](int k, int t, Weights& w) {
    const uint32_t past = k + 32 * piece < K ? 0u : 0x80000000u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(codes, (int)(wat[t][h] | past), k / 2, 0);
      w.c[h] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  };
  uint4 a[8];
  const int scale_stride = scale_row_bytes(K, 4 * kScaleWords);
  auto multiply = [&](int k, int t, const Weights& w) {
    uint32_t c[2][4] = {{w.c[0].x, w.c[0].y, w.c[0].z, w.c[0].w}, {w.c[1].x, w.c[1].y, w.c[1].z, w.c[1].w}};
#pragma unroll
    for (int j = 0; j < 4; ++j) halves(c[0][j], c[1][j]);
    transpose4(c[0]);
    transpose4(c[1]);
    uint32_t s[kScaleWords];
    __builtin_memcpy(s, __builtin_assume_aligned(shared + (t * 16 + col) * scale_stride + k / kGroup * kScaleBytes,
                                                 kScaleWords >= 4 ? 16 : 8),
                     4 * kScaleWords);
    if constexpr (kInt4) {
      // opaque to the compiler, so that each tile makes the offset's products anew: kept for all
      // tiles they would take 4 registers per 32 channels
      uint32_t c8 = 0xc100c100u;   // -8, -8
      asm volatile("" : "+v"(c8));
      const bf16x8 b8 = as_bf16x8(make_uint4(c8, c8, c8, c8));
      // the sums of up to four groups side by side, so that a product need not wait for the one before it: 32 rows
      // over 8 experts of 28672 x 7424, SiLU * up, take 429 / 260 / 242 us for groups of 32 / 64 / 128, one
      // group after the other 481 / 281 / 281
      constexpr int kGroups = kStep / kGroup, kSide = std::min(kGroups, 4);
#pragma unroll
      for (int g0 = 0; g0 < kGroups; g0 += kSide) {
        f32x4 d[kSide];
#pragma unroll
        for (int g = 0; g < kSide; ++g) d[g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < kGroup / 32; ++h)
#pragma unroll
          for (int g = 0; g < kSide; ++g) {
            const int j = (g0 + g) * (kGroup / 32) + h;
            d[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[j]), b8, d[g], 0, 0, 0);
            d[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[j]), as_bf16x8(unpack_int4(c[j >> 2][j & 3])), d[g], 0, 0, 0);
          }
#pragma unroll
        for (int g = 0; g < kSide; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(__uint_as_float(s[g0 + g]), d[g][i], acc[t][i]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            as_bf16x8(a[j]), as_bf16x8(unpack_mxfp4(c[j >> 2][j & 3], s[j >> 2] >> (8 * (j & 3)) & 0xff)), acc[t], 0, 0, 0);
    }
  };
  // every tile's weights of a step are in flight at once; a tile's next ones are asked for as
  // soon as it has been multiplied
  Weights w[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) load_weights(wave * kStep, t, w[t]);
  stage_scales<kInt4, kGroup, NT * 16>(
      static_cast<const uint8_t*>(p.scales) + (size_t)blk.e * p.N * (K / kGroup) * kScaleBytes,
      [&](int i) { return wrow(i >> 4, i & 15); }, K, shared);
  __syncthreads();
  for (int k = wave * kStep; k < K; k += kFbWaves * kStep) {
    // MFMA j has channels 32 j + 8 q onwards of the step; channels past K are zero
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = make_uint4(0, 0, 0, 0);
      if (k + 32 * j < K) a[j] = *reinterpret_cast<const uint4*>(ap + k + 32 * j + 8 * q);
      if constexpr (kInt4) a[j] = order_int4(a[j]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      multiply(k, t, w[t]);
      load_weights(k + kFbWaves * kStep, t, w[t]);   // past K: zeros, without a read
      __builtin_amdgcn_sched_barrier(0);   // a tile's temporaries end before the next tile's begin
    }
  }
  __syncthreads();   // the scales have been read
  const int rows = blk.hi - blk.lo;
  float* red = reinterpret_cast<float*>(shared);
  auto at = [&](int v, int t, int r, int c) { return ((v * NT + t) * BM + r) * 16 + c; };
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * q + i < rows) red[at(wave, t, 4 * q + i, col)] = acc[t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * kCols; i += kFbWaves * 64) {
    const int r = i / kCols, c = i % kCols;
    if (n0 + c >= n_out) continue;
    auto sum = [&](int t) {
      float s = red[at(0, t, r, c & 15)];
#pragma unroll
      for (int v = 1; v < kFbWaves; ++v) s += red[at(v, t, r, c & 15)];
      return s;
    };
    if constexpr (kSilu)
      store(blk.lo + r, n0 + c, silu_mul(sum(c / 16 * 2), sum(c / 16 * 2 + 1)));
    else
      store(blk.lo + r, n0 + c, sum(c / 16));
  }
}

// row blocks: at most one partial block per expert that has rows, and one of rows without an expert
static long long fourbit_blocks(long long M_rows, int E) {
  return std::min<long long>(M_rows, M_rows / 16 + std::min<long long>(E, M_rows) + 1);
}

// ---------------------------------------------------------------- rows of up to 7168 channels: streaming
//
// Bound by the weights' bytes from HBM: int4 groups of 128, 128 routes over 256 experts of 7168 x 2048
// take 166 us (789 MB, 4.8 TB/s); int4 groups of 32, 512 routes over 128 of 1536 x 2048, SiLU * up, 57
// (240 MB, 4.2; the VALU is busy 58% of the time, the MFMAs 15%); mxfp4, 64 routes over 8 of 28672 x 4096
// 103 (501 MB, 4.9).  One token on four experts of 5760 x 2880, mxfp4 (34 MB) is a chain: 1.8 us launch,
// 1.2 the experts' scan, 3.4 to the first item's arrival, then 1.7 to 2 us for each of two or three
// items: 13 us.  Each further 16 rows of an expert read and unpack its codes again: 16 / 32 / 64 rows for
// each of 32 experts of 5760 x 2880, SiLU * up, take 68 / 115 / 196 us in mxfp4, 102 / 168 / 309 in int4
// groups of 32.
//
// A launch is a fixed number of workgroups of eight waves.  Each takes an even share of the items
// (a block of up to 16 rows of one expert, 16 weight rows; with SiLU * up 8 gate and 8 up rows) in
// order, so that it reads consecutive weight rows, and streams them through a ring of LDS slots by
// direct loads of 1 KiB: all slots but one are in flight while one is multiplied, without a register
// for it.  Wave w has the activations of S steps of 128 channels in registers for as long as the
// row block lasts; the waves' f32 sums meet in LDS in wave order.  One barrier an item: behind it
// the next item's bytes have landed, the previous item's slot is free and its sums are complete.
//
// Not kept, being slower: workgroups of four waves, one workgroup per CU where two fit, items dealt
// to the workgroups in turn (174-265 us for 160), all slots filled before the first item instead of all
// but one (one token 14.1 us for 13.1).  More than 16 rows per expert: 32- and 64-row blocks in the
// other kernel, which read the weights fewer times, took 107 / 192 / 314 and 169 / 212 / 351 us at
// 16 / 32 / 64 rows per expert where this took 80 / 128 / 211 beside them (mxfp4, 32 experts, 5760 x 2880).
//
// A weight row's 16-byte pieces lie in its LDS row in the order piece ^ swizzle, chosen so that the
// 16 lanes that read one piece of 16 rows hit different banks.

constexpr int kStreamWaves = 8;
// steps a wave can hold activations for without spilling a register
constexpr int stream_max_steps(bool int4, int group) { return int4 && group == 32 ? 5 : 7; }

// the sum over the four rows of 16 lanes, in every lane
__device__ __forceinline__ float quads_total(float v) {
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// 16-byte pieces of a row of `pieces` are stored at piece ^ row_swizzle(pieces, row), row < 16: with
// G the largest power of two (to 16) in `pieces`, rows row + 16 / G start in the same bank, and
// differ by the swizzle within a group of G pieces
__device__ __forceinline__ int row_swizzle(int pieces, int row) {
  const int a = min(__builtin_ctz(pieces), 4);
  return row >> (4 - a) & ((1 << a) - 1);
}

template <bool kInt4, int kGroup, int S>
struct StreamCfg {
  static constexpr int W = kStreamWaves;
  static constexpr int kScaleBytes = kInt4 ? 4 : 1;
  static constexpr int kMaxK = W * S * 128;
  // KiB of LDS: one segment (8 rows) of codes and of scales
  static constexpr int kCodeKb = (8 * kMaxK / 2 + 1023) / 1024;
  static constexpr int kScaleKb = (8 * (kMaxK / kGroup) * kScaleBytes + (kInt4 ? 0 : 15) + 1023) / 1024;
  // runtime: the scales are copied from the aligned 16 bytes that hold their first one, so rows of
  // no whole 16 bytes take up to 15 more (int4's shorter rows are 4 bytes less each: still within kScaleKb)
  __device__ static int scale_kb(int row_bytes) { return (8 * row_bytes + (row_bytes % 16 ? 15 : 0) + 1023) / 1024; }
  static constexpr int kSlotKb = 2 * (kCodeKb + kScaleKb);
  static constexpr int kScaleLoads = (2 * kScaleKb + W - 1) / W;   // a wave's per item
  static constexpr int kLoads = S + kScaleLoads;
  static constexpr int kFixedKb = 2 * W + 1;   // two sets of sums, and a place for surplus loads
  // two workgroups per CU where two slots each fit in LDS and the loop in 128 registers (a spilled
  // register's reload would wait for the direct loads before it), else one
  static constexpr int kPerCu = 2 * (2 * kSlotKb + kFixedKb) <= 160 && S <= (kInt4 && kGroup == 32 ? 2 : 3) ? 2 : 1;
  static constexpr int kRingKb = 160 / kPerCu - kFixedKb;
  static constexpr int kMaxSlots = std::min(8, 63 / kLoads + 2);   // vmcnt counts to 63
  static_assert(kRingKb >= 2 * kSlotKb, "ring");
};

template <bool kInt4, int kGroup, bool kSilu, int S>
__global__ __launch_bounds__(kStreamWaves * 64, (StreamCfg<kInt4, kGroup, S>::kPerCu * 2)) void fourbit_stream_kernel(
    FourbitArgs p) {
  using Cfg = StreamCfg<kInt4, kGroup, S>;
  constexpr int W = kStreamWaves;
  constexpr int kRows = kSilu ? 8 : 16;   // output columns of an item
  constexpr int kGroups = S * 128 / kGroup, kSums = kInt4 ? (kGroups + 3) / 4 : 1;
  __shared__ __align__(16) uint8_t ring[Cfg::kRingKb * 1024];
  __shared__ __align__(16) uint8_t spare[1024];
  __shared__ float red[2][W][16][16];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int K = p.K;
  const int n_out = kSilu ? p.N / 2 : p.N;
  const int tiles = (n_out + kRows - 1) / kRows;
  auto store = [&](int r, int n, float v) {
    const size_t at = (size_t)r * n_out + n;
    if (p.c_f32)
      static_cast<float*>(p.C)[at] = v;
    else
      static_cast<uint16_t*>(p.C)[at] = f32_to_bf16_bits(v);
  };
  const RowBlocks rows_of(p.offsets, p.E, p.M_rows);
  // rows without an expert are zero
  {
    const int V = rows_of.at(p.E);
    const long long n = (long long)(p.M_rows - V) * n_out;
    for (long long i = (long long)blockIdx.x * W * 64 + threadIdx.x; i < n;
         i += (long long)gridDim.x * W * 64)
      store(V + (int)(i / n_out), (int)(i % n_out), 0.0f);
  }
  const int items = rows_of.count() * tiles;
  const int share = uniform(items / (int)gridDim.x), extra = items - share * (int)gridDim.x;
  const int first = (int)blockIdx.x * share + min((int)blockIdx.x, extra);
  const int n = uniform(share + ((int)blockIdx.x < extra ? 1 : 0));
  if (n == 0) return;

  // ---- this lane's part of the direct loads
  const int pieces = K / 32, row_bytes = K / 2;
  const int code_kb = (8 * row_bytes + 1023) / 1024;      // a segment's loads
  uint32_t code_at[S];                                     // source, from an item's first row
  int code_to[S];                                          // target, from the slot; < 0: the spare KiB
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const int load = wave * S + j, seg = (load >= code_kb) + (load >= 2 * code_kb);
    const int i = min((load - seg * code_kb) * 64 + lane, 8 * pieces - 1);   // piece of the segment, as it lies in LDS
    int r = 0;
#pragma unroll
    for (int m = 1; m < 8; ++m) r += i >= m * pieces;
    const int pos = i - r * pieces;
    const int row = kSilu ? min(r, n_out - 1) : min(seg * 8 + r, n_out - 1);
    code_at[j] = (uint32_t)(row + (kSilu ? seg * n_out : 0)) * (uint32_t)row_bytes +
                 (uint32_t)(pos ^ row_swizzle(pieces, seg * 8 + r)) * 16u;
    code_to[j] = seg < 2 ? seg * code_kb * 1024 + (load - seg * code_kb) * 1024 : -1;
    if (seg >= 2) code_at[j] = 0;
  }
  const int scale_row = K / kGroup * Cfg::kScaleBytes;     // bytes of scales of a weight row
  const int scale_pieces = scale_row % 16 == 0 ? scale_row / 16 : 1;   // odd rows are not swizzled
  const int rows0 = min(8, n_out);                         // rows of a segment that exist
  const int second = kSilu ? n_out : n_out > 8 ? 8 : 0;    // first row of the second segment
  const int rows1 = kSilu ? rows0 : max(min(8, n_out - 8), 1);
  const int scale_base = 2 * code_kb * 1024;
  const int scale_kb = Cfg::scale_kb(scale_row);
  const int slot_bytes = 2 * (code_kb + scale_kb) * 1024;
  const int slots = uniform(min(Cfg::kRingKb * 1024 / slot_bytes, Cfg::kMaxSlots));
  int scale_i[Cfg::kScaleLoads];                           // source piece
#pragma unroll
  for (int j = 0; j < Cfg::kScaleLoads; ++j) {
    const int load = wave * Cfg::kScaleLoads + j, seg = (load >= scale_kb) + (load >= 2 * scale_kb);
    const int i = (load - seg * scale_kb) * 64 + lane;
    int r = 0;
#pragma unroll
    for (int m = 1; m <= 8; ++m) r += i >= m * scale_pieces;
    scale_i[j] = i ^ (scale_row % 16 == 0 && r < 8 ? row_swizzle(scale_pieces, seg * 8 + r) : 0);
  }

  using Lds = __attribute__((address_space(3))) uint8_t*;
  const uint32_t ring_at = (uint32_t)(uintptr_t)(Lds)ring, spare_at = (uint32_t)(uintptr_t)(Lds)spare;
  // first weight row of a tile; the last tile of several reaches back to have all its rows
  auto row0_of = [&](int tile) { return max(min(tile * kRows, n_out - kRows), 0); };
  auto issue = [&](const RowBlock& b, int tile, int slot) {
    const size_t row = (size_t)b.e * p.N + row0_of(tile);
    const uint8_t* codes = uniform_ptr(p.codes + row * row_bytes);
    const uint32_t to = ring_at + slot * slot_bytes;
#pragma unroll
    for (int j = 0; j < S; ++j)
      dma16(uniform_u32(code_to[j] < 0 ? spare_at : to + code_to[j]), codes, code_at[j]);
#pragma unroll
    for (int j = 0; j < Cfg::kScaleLoads; ++j) {
      const int load = wave * Cfg::kScaleLoads + j, seg = (load >= scale_kb) + (load >= 2 * scale_kb);
      const uint8_t* from = static_cast<const uint8_t*>(p.scales) + (row + (seg == 1 ? second : 0)) * scale_row;
      const int shift = (int)(reinterpret_cast<uintptr_t>(from) & 15);
      const int end = (shift + (seg == 1 ? rows1 : rows0) * scale_row - 1) >> 4;   // last piece with a scale in it
      dma16(uniform_u32(seg < 2 ? to + scale_base + load * 1024 : spare_at), uniform_ptr(from - shift),
            (uint32_t)(seg < 2 ? min(scale_i[j], end) : 0) * 16u);
    }
  };

  // ---- this lane's part of the products
  const int wr = col & 7, wseg = col >> 3;
  int code_from[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int piece = min(4 * (wave * S + s) + q, pieces - 1);
    code_from[s] = wseg * code_kb * 1024 + wr * row_bytes + ((piece ^ row_swizzle(pieces, col)) << 4);
  }
  // int4: where a step's scales start (they lie in one 16-byte piece); mxfp4: each word
  constexpr int kFrom = kInt4 ? S : S + 1, kFromWords = kInt4 ? 128 / kGroup : 1;   // mxfp4's may start inside a word
  int scale_from[kFrom];
  const int scale_swz = scale_row % 16 == 0 ? row_swizzle(scale_pieces, col) : 0;
  const int scale_first = wave * (S * 128 / kGroup) * Cfg::kScaleBytes;   // byte of a row's scales
#pragma unroll
  for (int i = 0; i < kFrom; ++i) {
    const int b = scale_first + 4 * kFromWords * i;
    scale_from[i] = scale_base + wseg * scale_kb * 1024 + wr * scale_row + (((b >> 4) ^ scale_swz) << 4) + (b & 15);
  }
  // int4: this lane's scales as the offsets' second operand, group 4 i + q; groups of 32: word q of step i
  int sum_from[kInt4 && kGroup > 32 ? kSums : 1];
  if constexpr (kInt4 && kGroup > 32) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      const int b = scale_first + 4 * min(4 * i + q, kGroups - 1);
      sum_from[i] = scale_base + wseg * scale_kb * 1024 + wr * scale_row + (((b >> 4) ^ scale_swz) << 4) + (b & 15);
    }
  }
  uint32_t scale_ok[kInt4 ? 1 : S];   // mxfp4: bits of a step's word that are scales of channels below K
  if constexpr (!kInt4) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int there = scale_row - scale_first - 4 * s;
      scale_ok[s] = there >= 4 ? ~0u : there <= 0 ? 0u : (1u << (8 * there)) - 1;
    }
  }
  bf16x8 a[S][4];
  // int4: -8 times the sums of each group's activations, as the first operand of a 16x16x4 product
  // with the scales: lane 16 q + c has row c, group 4 i + q
  float sums[kSums];
  auto load_activations = [&](const RowBlock& b) {
    int r = min(b.lo + col, b.hi - 1);   // surplus rows repeat the last
    if (p.a_rows) r = min(max(p.a_rows[r] / p.a_div, 0), p.A_rows - 1);
    const uint16_t* ap = p.A + (size_t)r * K + 8 * q;
    uint4 raw[S][4];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = (wave * S + s) * 128 + 32 * j;
        raw[s][j] = make_uint4(0, 0, 0, 0);
        if (k < K) raw[s][j] = *reinterpret_cast<const uint4*>(ap + k);
      }
    if constexpr (kInt4)
#pragma unroll
      for (int i = 0; i < kSums; ++i) sums[i] = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kInt4) {
          float v[8], t = 0.0f;
          chunk_to_f32<uint16_t>(raw[s][j], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) t += v[i];
          const int g = (s * 128 + 32 * j) / kGroup;
          t = quads_total(t);
          sums[g / 4] += q == g % 4 ? -8.0f * t : 0.0f;
          raw[s][j] = order_int4(raw[s][j]);
        }
        // used here, so that the compiler waits for these loads here and not, with every direct
        // load, in front of each item's products
        asm volatile("" : "+v"(raw[s][j].x), "+v"(raw[s][j].y), "+v"(raw[s][j].z), "+v"(raw[s][j].w));
        a[s][j] = as_bf16x8(raw[s][j]);
      }
  };

  struct Cursor {
    int block, tile;
    RowBlock rows;
  };
  auto next = [&](Cursor& c) {
    c.tile = uniform(c.tile + 1);
    if (c.tile < tiles) return;
    c.tile = 0;
    c.block = uniform(c.block + 1);
    if (c.block < rows_of.count()) c.rows = rows_of.find(c.block);
  };
  const int first_block = uniform(first / tiles);
  Cursor load{first_block, uniform(first - first_block * tiles), rows_of.find(first_block)};
  Cursor cur = load, prev = load;
  for (int i = 0; i < min(n, slots - 1); ++i) {
    issue(load.rows, load.tile, i);
    next(load);
  }
  load_activations(cur.rows);
  int slot = 0, next_slot = slots - 1;
  // sums of an item, each wave's in turn to the front: rows * kRows outputs over the threads
  auto finish = [&](const Cursor& c, int i) {
    const int rows = c.rows.hi - c.rows.lo;
    const int o = (int)(threadIdx.x + (W - i % W) * 64) % (W * 64);
    if (o < rows * kRows) {
      const int r = o / kRows, n_at = o % kRows;
      auto sum = [&](int cc) {
        float s = red[i & 1][0][r][cc];
#pragma unroll
        for (int v = 1; v < W; ++v) s += red[i & 1][v][r][cc];
        return s;
      };
      float v = sum(n_at);
      if constexpr (kSilu) v = silu_mul(v, sum(8 + n_at));
      const int row = row0_of(c.tile) + n_at;
      if (row >= c.tile * kRows && row < n_out) store(c.rows.lo + r, row, v);   // overlapped columns: the tile before
    }
  };
  for (int i = 0; i < n; ++i) {
    // loads of this item have landed; LDS is drained: everyone's reads of the previous slot and
    // writes of sums are behind the barrier
    wait_slices<Cfg::kLoads, Cfg::kMaxSlots - 2, true>(min(slots - 2, n - 1 - i));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (i + slots - 1 < n) {
      issue(load.rows, load.tile, next_slot);
      next(load);
    }
    next_slot = next_slot + 1 == slots ? 0 : next_slot + 1;
    if (i > 0) finish(prev, i - 1);
    const uint8_t* in = ring + slot * slot_bytes;
    slot = slot + 1 == slots ? 0 : slot + 1;
    // scales
    uint32_t shift = 0;   // bytes before the first scale (rows that are not swizzled)
    if (scale_row % 16 != 0)
      shift = (uint32_t)((reinterpret_cast<uintptr_t>(p.scales) +
                          ((size_t)cur.rows.e * p.N + row0_of(cur.tile) + (wseg ? second : 0)) * scale_row) & 15);
    uint32_t sc[kInt4 ? 1 : S];   // mxfp4: a step's four bytes
    if constexpr (!kInt4) {
      const uint32_t odd = (scale_from[0] + shift) & 3;   // the same for every word
      uint32_t raw[S + 1];
#pragma unroll
      for (int w = 0; w <= S; ++w) raw[w] = *reinterpret_cast<const uint32_t*>(in + ((scale_from[w] + shift) & ~3u));
#pragma unroll
      for (int w = 0; w < S; ++w)   // past K: 2^0
        sc[w] = (__builtin_amdgcn_alignbyte(raw[w + 1], raw[w], odd) & scale_ok[w]) | (0x7f7f7f7fu & ~scale_ok[w]);
    }
    // two sums, so that a product need not wait for the one before it
    f32x4 acc[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if constexpr (kInt4) {
        // the offsets of four groups, in front of their products: the sums stay small (all offsets first
        // would have them start from minus the whole row's)
        if (s % (kGroup / 32) == 0) {
          const int i = s / (kGroup / 32), g = 4 * i + q;
          const int from = kGroup > 32 ? sum_from[kGroup > 32 ? i : 0] : scale_from[kGroup > 32 ? 0 : i] + 4 * q;
          const float f = *reinterpret_cast<const float*>(in + from + shift);
          const bool there = g < kGroups && wave * S * 128 + g * kGroup < K;
          acc[i & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(sums[i], there ? f : 0.0f, acc[i & 1], 0, 0, 0);
        }
      }
      const uint4 v = *reinterpret_cast<const uint4*>(in + code_from[s]);
      uint32_t c[4] = {v.x, v.y, v.z, v.w};
      transpose4(c);
      if constexpr (kInt4) {
        float f[128 / kGroup];   // past K: 0
#pragma unroll
        for (int i = 0; i < 128 / kGroup; ++i) {
          f[i] = *reinterpret_cast<const float*>(in + scale_from[s] + shift + 4 * i);
          if ((wave * S + s) * 128 + i * kGroup >= K) f[i] = 0.0f;
        }
        f32x4 d;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (32 * j % kGroup == 0) d = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[s][j], as_bf16x8(unpack_int4(c[j])), d, 0, 0, 0);
          if (32 * (j + 1) % kGroup == 0)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[j & 1][e] = fmaf(f[32 * j / kGroup], d[e], acc[j & 1][e]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[j & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a[s][j], as_bf16x8(unpack_mxfp4(c[j], sc[s] >> (8 * j) & 0xff)), acc[j & 1], 0, 0, 0);
      }
    }
    const int rows = cur.rows.hi - cur.rows.lo;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (4 * q + e < rows) red[i & 1][wave][4 * q + e][col] = acc[0][e] + acc[1][e];
    prev = cur;
    next(cur);
    if (cur.block != prev.block && i + 1 < n) load_activations(cur.rows);
  }
  __syncthreads();
  finish(prev, n - 1);
}

// How a launch is cut: the streaming kernel where its waves hold the activations of a whole row,
// else NT weight tiles a workgroup.
struct FourbitCut {
  bool stream;
  int NT;
  long long lds;          // dynamic LDS bytes of a workgroup
  long long workgroups;   // streaming: items
};

constexpr int kMaxLds = 64 << 10;   // dynamic LDS of a launch

static FourbitCut fourbit_cut(long long M_rows, int E, long long n_out, long long K, bool int4, int group, bool silu) {
  FourbitCut c{};
  if (K <= kStreamWaves * stream_max_steps(int4, group) * 128) {
    c.stream = true;
    c.workgroups = fourbit_blocks(M_rows, E) * ((n_out + (silu ? 7 : 15)) / (silu ? 8 : 16));
    return c;
  }
  const int per = silu ? 2 : 1;   // weight tiles of an output tile
  const int step_bytes = kStep / group * (int4 ? 4 : 1);
  // the scales of the tiles' rows; afterwards the waves' sums
  const auto lds = [&](int nt) {
    return std::max<long long>((long long)nt * 16 * scale_row_bytes(K, step_bytes), kFbWaves * nt * 1024);
  };
  c.NT = 4;
  while (c.NT > per && lds(c.NT) > kMaxLds) c.NT /= 2;
  c.lds = lds(c.NT);
  c.workgroups = fourbit_blocks(M_rows, E) * ((n_out + 16 * (c.NT / per) - 1) / (16 * (c.NT / per)));
  return c;
}

bool fourbit_fits(long long M_rows, int E, long long N, long long K, bool int4, int group, bool silu) {
  if (M_rows > INT_MAX - 64) return false;   // the kernels count up to a block past the rows in 32 bits
  const FourbitCut c = fourbit_cut(M_rows, E, silu ? N / 2 : N, K, int4, group, silu);
  // a grid holds fewer than 2^32 threads; items are counted in 32 bits
  return c.stream ? c.workgroups <= INT_MAX : c.workgroups < (1ll << 24) && c.lds <= kMaxLds;
}

template <bool kInt4, int kGroup, bool kSilu>
static hipError_t launch_fourbit_stream(const FourbitArgs& a, long long items, hipStream_t stream) {
  const int steps = (a.K + 127) / 128;
  const auto go = [&](auto s) {
    constexpr int S = decltype(s)::value;
    const unsigned grid = (unsigned)std::min<long long>(items, 256 * StreamCfg<kInt4, kGroup, S>::kPerCu);
    hipLaunchKernelGGL((fourbit_stream_kernel<kInt4, kGroup, kSilu, S>), dim3(grid), dim3(kStreamWaves * 64), 0, stream, a);
    return hipGetLastError();
  };
  const int S = (steps + kStreamWaves - 1) / kStreamWaves;
  if (S == 1) return go(std::integral_constant<int, 1>{});
  if (S == 2) return go(std::integral_constant<int, 2>{});
  if (S == 3) return go(std::integral_constant<int, 3>{});
  if (S == 4) return go(std::integral_constant<int, 4>{});
  if (S == 5) return go(std::integral_constant<int, 5>{});
  if constexpr (stream_max_steps(kInt4, kGroup) > 5) {
    if (S == 6) return go(std::integral_constant<int, 6>{});
    if (S == 7) return go(std::integral_constant<int, 7>{});
  }
  return hipErrorInvalidValue;
}

template <bool kInt4, int kGroup, bool kSilu>
static hipError_t launch_fourbit_s(const FourbitLaunch& p, hipStream_t stream) {
  const FourbitCut cut =
      fourbit_cut(p.M_rows, p.E, kSilu ? p.N / 2 : p.N, p.K, kInt4, kGroup, kSilu);
  const FourbitArgs a{static_cast<const uint16_t*>(p.A), p.a_rows, p.a_div, (int)p.a_total,
                      static_cast<const uint8_t*>(p.codes), p.scales, p.offsets, p.E, (int)p.M_rows, (int)p.N,
                      (int)p.K, p.C, p.c_f32};
  if (cut.stream) return launch_fourbit_stream<kInt4, kGroup, kSilu>(a, cut.workgroups, stream);
  const dim3 grid((unsigned)cut.workgroups), block(kFbWaves * 64);
#define MOE_FOURBIT(NT_)                                                                                    \
  if (cut.NT == NT_) {                                                                                      \
    hipLaunchKernelGGL((fourbit_kernel<kInt4, kGroup, kSilu, NT_>), grid, block, (size_t)cut.lds, stream, a); \
    return hipGetLastError();                                                                               \
  }
  if constexpr (!kSilu) { MOE_FOURBIT(1) }
  MOE_FOURBIT(2)
  MOE_FOURBIT(4)
#undef MOE_FOURBIT
  return hipErrorInvalidValue;
}

template <bool kInt4, int kGroup>
static hipError_t launch_fourbit_g(const FourbitLaunch& p, hipStream_t stream) {
  return p.silu ? launch_fourbit_s<kInt4, kGroup, true>(p, stream) : launch_fourbit_s<kInt4, kGroup, false>(p, stream);
}

hipError_t launch_fourbit(const FourbitLaunch& p, hipStream_t stream) {
  if (p.M_rows <= 0) return hipSuccess;
  if (!p.int4) return launch_fourbit_g<false, 32>(p, stream);
  if (p.group == 32) return launch_fourbit_g<true, 32>(p, stream);
  if (p.group == 64) return launch_fourbit_g<true, 64>(p, stream);
  return launch_fourbit_g<true, 128>(p, stream);
}

// Quantises groups of kGroup consecutive channels, eight channels a lane.
//   int4:  scale = amax / 7 (1 if that is zero), code = 8 + round(w / scale)
//   mxfp4: scale = 2^(floor(log2 amax) - 2), code = w / scale in e2m1; ties to the even code,
//          magnitudes past 6 give 6
// Bound by HBM: 32 x 5760 x 2880 to mxfp4 takes 337 us from bf16 (1.34 GB, 4.0 TB/s), 411 from f32 (2.40 GB,
// 5.8); x 2816 to int4 groups of 128 333 and 399.
template <bool kInt4, int kGroup, bool kBf16In>
__global__ __launch_bounds__(256) void quantize_fourbit_kernel(const void* __restrict__ w_, long long n8,
                                                               uint32_t* __restrict__ codes, void* __restrict__ scales) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;   // n8 % (kGroup / 8) == 0: groups are whole
  if (i >= n8) return;
  float v[8];
  if constexpr (kBf16In) {
    chunk_to_f32<uint16_t>(static_cast<const uint4*>(w_)[i], v);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[4];
      chunk_to_f32<float>(static_cast<const uint4*>(w_)[2 * i + h], f);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * h + j] = f[j];
    }
  }
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
#pragma unroll
  for (int o = 1; o < kGroup / 8; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, kWave));
  const bool first = i % (kGroup / 8) == 0;
  const long long group = i / (kGroup / 8);
  uint32_t out = 0;
  if constexpr (kInt4) {
    float s = amax / 7.0f;
    if (s == 0.0f) s = 1.0f;
    if (first) static_cast<float*>(scales)[group] = s;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      out |= (uint32_t)((int)fminf(fmaxf(rintf(v[j] / s), -8.0f), 7.0f) + 8) << (4 * j);
  } else {
    // exponent field of amax (a subnormal counts as the smallest), less the 2 of e2m1's 4 = 2^2
    const int ex = (int)(__float_as_uint(amax) >> 23 & 0xff);
    const int s = amax == 0.0f ? 127 : min(max(ex - 2, 0), 254);
    if (first) static_cast<uint8_t*>(scales)[group] = (uint8_t)s;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = ldexpf(fabsf(v[j]), 127 - s);
      const uint32_t mag = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
      out |= (mag | (__float_as_uint(v[j]) >> 31 << 3)) << (4 * j);
    }
  }
  codes[i] = out;
}

template <bool kInt4, int kGroup>
static hipError_t launch_quantize_g(const void* w, bool bf16, long long n, void* codes, void* scales, hipStream_t stream) {
  const long long n8 = n / 8;
  const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
  if (bf16)
    hipLaunchKernelGGL((quantize_fourbit_kernel<kInt4, kGroup, true>), grid, block, 0, stream, w, n8,
                       static_cast<uint32_t*>(codes), scales);
  else
    hipLaunchKernelGGL((quantize_fourbit_kernel<kInt4, kGroup, false>), grid, block, 0, stream, w, n8,
                       static_cast<uint32_t*>(codes), scales);
  return hipGetLastError();
}

hipError_t launch_quantize_fourbit(const void* w, bool bf16, long long n, bool int4, int group, void* codes,
                                   void* scales, hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  if (!int4) return launch_quantize_g<false, 32>(w, bf16, n, codes, scales, stream);
  if (group == 32) return launch_quantize_g<true, 32>(w, bf16, n, codes, scales, stream);
  if (group == 64) return launch_quantize_g<true, 64>(w, bf16, n, codes, scales, stream);
  return launch_quantize_g<true, 128>(w, bf16, n, codes, scales, stream);
}

}  // namespace moe
