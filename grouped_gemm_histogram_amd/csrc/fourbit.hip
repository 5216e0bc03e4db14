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

// eight e2m1 codes -> bf16 code * scale, in channel order
__device__ __forceinline__ uint4 unpack_mxfp4(uint32_t v, float scale) {
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3));
  return r;
}

// An e8m0 byte as f32: 2^(b - 127); 0 is 2^-127, 255 is NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
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
};

// kGroup: channels per scale (mxfp4: 32).  kTiles column tiles of a wave: gate and up, or one.
template <bool kInt4, int kGroup, bool kSilu, int MT, bool kF32Out, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void fourbit_kernel(FourbitArgs p) {
  constexpr int kTiles = kSilu ? 2 : 1;
  constexpr int BM = 16 * MT;
  __shared__ float red[kWaves][MT][kTiles][16][16];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int col = lane & 15, q = lane >> 4;
  const int n_out = kSilu ? p.N / 2 : p.N;
  const int tiles = (n_out + 15) / 16;
  const int n0 = (int)(blockIdx.x % tiles) * 16;
  const RowBlock blk = find_block(p.offsets, p.E, p.M_rows, BM, blockIdx.x / tiles);
  auto store = [&](int r, int n, float v) {
    const size_t at = (size_t)r * n_out + n;
    if constexpr (kF32Out)
      static_cast<float*>(p.C)[at] = v;
    else
      static_cast<uint16_t*>(p.C)[at] = f32_to_bf16_bits(v);
  };
  if (blk.e < 0) {   // rows without an expert are zero
    for (int i = threadIdx.x; i < (blk.hi - blk.lo) * 16; i += kWaves * 64)
      if (n0 + (i & 15) < n_out) store(blk.lo + (i >> 4), n0 + (i & 15), 0.0f);
    return;
  }
  const int K = p.K;
  // this lane's column of each tile and its row of each row tile (surplus ones repeat the last)
  const uint8_t* wp[kTiles];
  const uint8_t* sp[kTiles];
  constexpr int kScaleBytes = kInt4 ? 4 : 1;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const size_t n = (size_t)blk.e * p.N + (size_t)t * n_out + min(n0 + col, n_out - 1);
    wp[t] = p.codes + n * (K / 2);
    sp[t] = static_cast<const uint8_t*>(p.scales) + n * (K / kGroup) * kScaleBytes;
  }
  const uint16_t* ap[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    int r = min(blk.lo + m * 16 + col, blk.hi - 1);
    if (p.a_rows) r = min(max(p.a_rows[r] / p.a_div, 0), p.A_rows - 1);
    ap[m] = p.A + (size_t)r * K;
  }
  f32x4 acc[MT][kTiles];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // a step is 128 channels: 16 bytes of codes a lane and tile
  for (int k0 = wave * 128; k0 < K; k0 += kWaves * 128) {
    const bool mine = k0 + 32 * q < K;   // K % 32 == 0: a lane's 32 channels are all in the row or none
    uint32_t w[kTiles][4];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (mine) v = *reinterpret_cast<const uint4*>(wp[t] + (k0 + 32 * q) / 2);
      w[t][0] = v.x; w[t][1] = v.y; w[t][2] = v.z; w[t][3] = v.w;
    }
    if constexpr (kInt4) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t) transpose4(w[t]);
      f32x4 d[MT][kTiles];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (k0 + 32 * j >= K) break;
        if (32 * j % kGroup == 0)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < kTiles; ++t) d[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const bf16x8 a = as_bf16x8(order_int4(*reinterpret_cast<const uint4*>(ap[m] + k0 + 32 * j + 8 * q)));
          const uint32_t c136 = 0xc308c308u;
          const f32x4 off = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a, as_bf16x8(make_uint4(c136, c136, c136, c136)), f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
            d[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, as_bf16x8(unpack_int4(w[t][j])), d[m][t] + off, 0, 0, 0);
        }
        if (32 * (j + 1) % kGroup == 0 || k0 + 32 * (j + 1) >= K) {
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            const float s = reinterpret_cast<const float*>(sp[t])[(k0 + 32 * j) / kGroup];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[m][t][i] = fmaf(s, d[m][t][i], acc[m][t][i]);
          }
        }
      }
    } else {
      float s[kTiles];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) s[t] = mine ? e8m0_to_f32(sp[t][k0 / 32 + q]) : 1.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 b[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) b[t] = as_bf16x8(unpack_mxfp4(w[t][j], s[t]));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (mine) v = *reinterpret_cast<const uint4*>(ap[m] + k0 + 32 * q + 8 * j);
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
            acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(v), b[t], acc[m][t], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][m][t][4 * q + i][col] = acc[m][t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < BM * 16; i += kWaves * 64) {
    const int r = i >> 4, c = i & 15;
    float s[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      s[t] = red[0][r >> 4][t][r & 15][c];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) s[t] += red[v][r >> 4][t][r & 15][c];
    }
    if (blk.lo + r < blk.hi && n0 + c < n_out) {
      float out = s[0];
      if constexpr (kSilu) out = silu_mul(s[0], s[kTiles - 1]);
      store(blk.lo + r, n0 + c, out);
    }
  }
}

// row blocks: at most one partial block per expert that has rows, and one of rows without an expert
static long long fourbit_blocks(long long M_rows, int E, int BM) {
  return std::min<long long>(M_rows, M_rows / BM + std::min<long long>(E, M_rows) + 1);
}

// row tiles of 16 per row block
static int fourbit_row_tiles(long long M_rows, int E) { return M_rows <= 8ll * E ? 1 : 4; }

long long fourbit_workgroups(long long M_rows, int E, long long n_out) {
  return (n_out + 15) / 16 * fourbit_blocks(M_rows, E, 16 * fourbit_row_tiles(M_rows, E));
}

template <bool kInt4, int kGroup, bool kSilu, int MT>
static hipError_t launch_fourbit_t(const FourbitLaunch& p, hipStream_t stream) {
  constexpr int kWaves = 4;
  constexpr int BM = 16 * MT;
  const int n_out = (int)(kSilu ? p.N / 2 : p.N);
  const long long blocks = fourbit_blocks(p.M_rows, p.E, BM);
  FourbitArgs a{static_cast<const uint16_t*>(p.A), p.a_rows, p.a_div, (int)p.a_total,
                static_cast<const uint8_t*>(p.codes), p.scales, p.offsets, p.E, (int)p.M_rows, (int)p.N, (int)p.K, p.C};
  const dim3 grid((unsigned)((n_out + 15) / 16 * blocks)), block(kWaves * 64);
  if (p.c_f32)
    hipLaunchKernelGGL((fourbit_kernel<kInt4, kGroup, kSilu, MT, true, kWaves>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((fourbit_kernel<kInt4, kGroup, kSilu, MT, false, kWaves>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <bool kInt4, int kGroup>
static hipError_t launch_fourbit_g(const FourbitLaunch& p, hipStream_t stream) {
  const bool one = fourbit_row_tiles(p.M_rows, p.E) == 1;
  if (p.silu) return one ? launch_fourbit_t<kInt4, kGroup, true, 1>(p, stream) : launch_fourbit_t<kInt4, kGroup, true, 4>(p, stream);
  return one ? launch_fourbit_t<kInt4, kGroup, false, 1>(p, stream) : launch_fourbit_t<kInt4, kGroup, false, 4>(p, stream);
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
