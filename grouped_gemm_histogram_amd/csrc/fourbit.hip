// fourbit.hip -- grouped products with 4-bit weights and group scales, for few rows per expert:
//
//   C[p, n] = sum_k A[row(p), k] * W[e(p), n, k]         (optionally silu(gate) * up)
//
// int4: W = (code - 8) * scale, f32 scales per 32, 64 or 128 channels.  mxfp4: W = e2m1(code) *
// 2^(scale - 127), one e8m0 byte per 32 channels.  Codes are [E, N, K/2], the even channel in the
// low nibble.
//
// A workgroup has up to 16 * MT rows of one expert and 16 columns (with SiLU * up: 16 gate and
// 16 up columns); its waves split K and join their f32 sums in LDS in wave order.  A lane loads
// 16 bytes of codes, 32 channels of one column, and turns them into bf16 MFMA operands in
// registers: the sixteen rows of v_mfma_f32_16x16x32_bf16 make the product free at any row
// count, the weights' bytes bound it.
//
// mxfp4: e2m1 * 2^s is exact in bf16, so the scale is applied while unpacking
// (v_cvt_scalef32_pk_bf16_fp4); the four channel octets of a lane go to four MFMAs.
// int4: code * scale is not exact in bf16, so the MFMA runs on 128 + code (the nibble put under
// bf16's 128) and the scale multiplies its f32 result: the four lane groups first swap 4 x 4
// words (v_permlane32_swap, v_permlane16_swap) so that an MFMA has 32 consecutive channels, all
// of one scale.  The offset 136 leaves through a second MFMA with the constant weight -136,
// shared by gate and up.  Its terms are at most 17 times the true ones, 2^-24 each.

#include <algorithm>
#include <type_traits>

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

// eight int4 codes -> bf16 128 + code, in the channel order 0 4 1 5 2 6 3 7
__device__ __forceinline__ uint4 unpack_int4(uint32_t v) {
  return make_uint4((v & 0x000f000fu) | 0x43004300u, ((v >> 4) & 0x000f000fu) | 0x43004300u,
                    ((v >> 8) & 0x000f000fu) | 0x43004300u, ((v >> 12) & 0x000f000fu) | 0x43004300u);
}

// eight activations into the same order
__device__ __forceinline__ uint4 order_int4(uint4 a) {
  return make_uint4(__builtin_amdgcn_perm(a.z, a.x, 0x05040100u), __builtin_amdgcn_perm(a.z, a.x, 0x07060302u),
                    __builtin_amdgcn_perm(a.w, a.y, 0x05040100u), __builtin_amdgcn_perm(a.w, a.y, 0x07060302u));
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

// Where row block `block` of a launch lies: rows [lo, hi) of expert e, or with e < 0 rows
// [lo, hi) past the last valid row.  Every lane gets the result; all 64 lanes take part.
struct RowBlock {
  int e, lo, hi;
};

__device__ __forceinline__ RowBlock find_block(const int* __restrict__ offsets, int E, int M_rows, int BM, int block) {
  const int lane = lane_id();
  const int per = (E + kWave - 1) / kWave;   // consecutive experts per lane
  auto at = [&](int e) { return min(max(offsets[min(e, E)], 0), M_rows); };
  int mine = 0;
  for (int i = 0, lo = at(lane * per); i < per; ++i) {
    const int hi = at(lane * per + i + 1);
    mine += max(hi - lo + BM - 1, 0) / BM;
    lo = hi;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int up = __shfl_up(incl, o, kWave);
    if (lane >= o) incl += up;
  }
  const uint64_t below = __ballot(incl > block);
  if (below == 0) {   // past the experts' blocks: rows without an expert
    const int total = __builtin_amdgcn_readlane(incl, 63);
    const int V = at(E);
    const long long lo = V + (long long)(block - total) * BM;
    RowBlock r{-1, M_rows, M_rows};
    if (lo < M_rows) r = {-1, (int)lo, min((int)lo + BM, M_rows)};
    return r;
  }
  const int owner = __builtin_ctzll(below);
  int rest = block - (__shfl(incl, owner, kWave) - __shfl(mine, owner, kWave));
  RowBlock r{-1, M_rows, M_rows};
  for (int i = 0, lo = at(owner * per); i < per; ++i) {
    const int hi = at(owner * per + i + 1);
    const int nb = max(hi - lo + BM - 1, 0) / BM;
    if (rest < nb) {
      r = {owner * per + i, lo + rest * BM, min(lo + (rest + 1) * BM, hi)};
      break;
    }
    rest -= nb;
    lo = hi;
  }
  return r;
}

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

#ifndef FB_WAVES
#define FB_WAVES 4
#define FB_NT 4
#define FB_WG 512
#endif
constexpr int kFbWaves = FB_WAVES;
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

// kGroup: channels per scale (mxfp4: 32).  MT row tiles, NT weight tiles of 16 rows (with SiLU * up
// the even ones are gate and the odd ones up).
template <bool kInt4, int kGroup, bool kSilu, int MT, int NT>
__global__ __launch_bounds__(kFbWaves * 64, 2) void fourbit_kernel(FourbitArgs p) {
  constexpr int BM = 16 * MT;
  constexpr int kCols = (kSilu ? NT / 2 : NT) * 16;   // output columns
  constexpr int kScaleBytes = kInt4 ? 4 : 1;
  constexpr int kScaleWords = kStepScaleBytes<kInt4, kGroup> / 4;   // scales of a row per step
  // the scales of all tiles' rows, and after the loop the waves' sums [wave][tile][row][16]
  extern __shared__ __align__(16) uint8_t shared[];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int n_out = kSilu ? p.N / 2 : p.N;
  const int groups = (n_out + kCols - 1) / kCols;
  const int n0 = (int)(blockIdx.x % groups) * kCols;
  const RowBlock blk = find_block(p.offsets, p.E, p.M_rows, BM, blockIdx.x / groups);
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
  const uint16_t* ap[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    int r = min(blk.lo + m * 16 + col, blk.hi - 1);
    if (p.a_rows) r = min(max(p.a_rows[r] / p.a_div, 0), p.A_rows - 1);
    ap[m] = p.A + (size_t)r * K;
  }
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

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
  uint4 a[MT][8];
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
      uint32_t c136 = 0xc308c308u;
      asm volatile("" : "+v"(c136));
      const bf16x8 b136 = as_bf16x8(make_uint4(c136, c136, c136, c136));
      f32x4 d[MT];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bf16x8 b = as_bf16x8(unpack_int4(c[j >> 2][j & 3]));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (32 * j % kGroup == 0) d[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          d[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[m][j]), b136, d[m], 0, 0, 0);
          d[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[m][j]), b, d[m], 0, 0, 0);
          if (32 * (j + 1) % kGroup == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][t][i] = fmaf(__uint_as_float(s[32 * j / kGroup]), d[m][i], acc[m][t][i]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bf16x8 b = as_bf16x8(unpack_mxfp4(c[j >> 2][j & 3], s[j >> 2] >> (8 * (j & 3)) & 0xff));
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[m][j]), b, acc[m][t], 0, 0, 0);
      }
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
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[m][j] = make_uint4(0, 0, 0, 0);
        if (k + 32 * j < K) a[m][j] = *reinterpret_cast<const uint4*>(ap[m] + k + 32 * j + 8 * q);
        if constexpr (kInt4) a[m][j] = order_int4(a[m][j]);
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
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (m * 16 + 4 * q + i < rows) red[at(wave, t, m * 16 + 4 * q + i, col)] = acc[m][t][i];
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
static long long fourbit_blocks(long long M_rows, int E, int BM) {
  return std::min<long long>(M_rows, M_rows / BM + std::min<long long>(E, M_rows) + 1);
}

// How a launch is cut: row tiles per row block by the rows an expert has on average, weight tiles
// per workgroup by how many workgroups that leaves.
constexpr int kMaxNT = FB_NT, kMinWg = FB_WG;

struct FourbitCut {
  int MT, NT;
  long long workgroups;
};

static FourbitCut fourbit_cut(long long M_rows, int E, long long n_out, bool silu) {
  FourbitCut c;
  c.MT = M_rows <= 8ll * E ? 1 : M_rows <= 24ll * E ? 2 : 4;
  const long long blocks = fourbit_blocks(M_rows, E, 16 * c.MT);
  const auto wgs = [&](int nt) { return blocks * ((n_out + 16 * nt - 1) / (16 * nt)); };
  int nt = c.MT == 4 ? 1 : silu || c.MT == 2 ? kMaxNT / 2 : kMaxNT;   // output tiles
  if (c.MT == 2 && silu) nt = kMaxNT / 4;
  if (c.MT == 1)
    while (nt > 1 && wgs(nt) < kMinWg) nt /= 2;
  c.NT = silu ? 2 * nt : nt;
  c.workgroups = wgs(nt);
  return c;
}

// the scales of the tiles' rows; afterwards the waves' sums
static int fourbit_lds(int MT, int NT, long long K, int step_bytes) {
  return std::max(NT * 16 * scale_row_bytes(K, step_bytes), kFbWaves * NT * MT * 1024);
}

long long fourbit_workgroups(long long M_rows, int E, long long n_out, bool silu) {
  return fourbit_cut(M_rows, E, n_out, silu).workgroups;
}

template <bool kInt4, int kGroup, bool kSilu>
static hipError_t launch_fourbit_s(const FourbitLaunch& p, hipStream_t stream) {
  const FourbitCut cut = fourbit_cut(p.M_rows, p.E, kSilu ? p.N / 2 : p.N, kSilu);
  const FourbitArgs a{static_cast<const uint16_t*>(p.A), p.a_rows, p.a_div, (int)p.a_total,
                      static_cast<const uint8_t*>(p.codes), p.scales, p.offsets, p.E, (int)p.M_rows, (int)p.N,
                      (int)p.K, p.C, p.c_f32};
  const dim3 grid((unsigned)cut.workgroups), block(kFbWaves * 64);
  const int lds = fourbit_lds(cut.MT, cut.NT, p.K, kStepScaleBytes<kInt4, kGroup>);
  constexpr int kPer = kSilu ? 2 : 1;   // weight tiles per output tile
#define MOE_FOURBIT(MT_, NT_)                                                                             \
  if (cut.MT == MT_ && cut.NT == NT_ * kPer) {                                                            \
    hipLaunchKernelGGL((fourbit_kernel<kInt4, kGroup, kSilu, MT_, NT_ * kPer>), grid, block, lds, stream, a); \
    return hipGetLastError();                                                                               \
  }
  MOE_FOURBIT(1, 1)
  if constexpr (kMaxNT >= 4 || !kSilu) { MOE_FOURBIT(1, 2) }
  if constexpr (kMaxNT / kPer >= 4) { MOE_FOURBIT(1, 4) }
  if constexpr (kMaxNT / kPer >= 8) { MOE_FOURBIT(1, 8) }
  MOE_FOURBIT(2, (kMaxNT / 2 / kPer))
  MOE_FOURBIT(4, 1)
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
