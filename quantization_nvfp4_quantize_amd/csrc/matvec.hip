// Products of a few tokens with 4-bit weights on gfx950: y[m][n] = gs * sum_k
// x[m][k] * e2m1(w[n][k]) * scale[n][k / g], x bf16, W NVFP4 (E4M3 scale per 16,
// fp32 tensor scale) or MXFP4 (E8M0 scale per 32).
//
// e2m1 * scale has at most 6 significant bits for E4M3 and 2 for E8M0, so every
// weight is a bf16 value exactly, every product is exact and the matrix cores
// accumulate in fp32; the tensor scale multiplies the sum.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gemm_common.hpp"
#include "launch.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct MatvecParams {
  const uint16_t* x;    // bf16 [M][K]
  const uint8_t* w_q;   // [N][K/2]
  const uint8_t* w_s;   // [N][K/16] or [N][K/32]
  const float* w_gs;    // NVFP4 only
  void* out;            // [M][N]
  int64_t M, N;
  int K;
  bool bf16_out;
};

constexpr int kMvStep = 128;  // K per step: 64 bytes of a row of W, 16 of each of 4 lanes

// 8 nibbles of one dword times a scale -> 8 bf16, exact.
template <int FMT>
__device__ __forceinline__ bf16x8 weights8(uint32_t q, float s) {
  bf16x8 v;
  if constexpr (FMT == kMxfp4) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3);
    v = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
    v = bf16x8{(__bf16)(a[0] * s), (__bf16)(a[1] * s), (__bf16)(b[0] * s), (__bf16)(b[1] * s),
               (__bf16)(c[0] * s), (__bf16)(c[1] * s), (__bf16)(d[0] * s), (__bf16)(d[1] * s)};
  }
  return v;
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), b, c, 0, 0, 0);
}

// The 4 x 4 exchange of dwords between the four rows of 16 lanes: dword t of
// lane row s becomes dword s of lane row t.
__device__ __forceinline__ u32x4 exchange(u32x4 w) {
  const auto a = __builtin_amdgcn_permlane16_swap(w.x, w.y, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(w.z, w.w, false, false);
  const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  return u32x4{c[0], d[0], c[1], d[1]};
}

// Orders a wave's LDS traffic between its lanes.  (The hardware keeps it in
// order; this keeps the compiler to it.)
__device__ __forceinline__ void wave_sync() {
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ void store_result(const MatvecParams& p, int64_t m, int64_t n, float v) {
  if (m >= p.M || n >= p.N) return;
  if (p.bf16_out) static_cast<__bf16*>(p.out)[m * p.N + n] = (__bf16)v;
  else static_cast<float*>(p.out)[m * p.N + n] = v;
}

// Dwords of scales per row and step of 128 k.
template <int FMT>
constexpr int kUnit = FMT == kNvfp4 ? 2 : 1;

// The scales of one step for ROWS rows of W, `stride` bytes apart but none
// behind the last, into LDS rows `out_stride` dwords apart.  Of the row's last,
// partial step only the first `blocks` 32-k blocks exist; the others are 0.
template <int FMT, int ROWS>
__device__ __forceinline__ void stage_step(const uint8_t* src, int row, int row_step, int rows, size_t stride, int blocks,
                                           uint32_t* out, int out_stride) {
  constexpr int kBytes = 4 * kUnit<FMT>;
  uint32_t v[ROWS][kUnit<FMT>];
  if (blocks >= 4) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) __builtin_memcpy(v[r], src + (size_t)min(row + r * row_step, rows - 1) * stride, kBytes);
  } else {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const uint8_t* at = src + (size_t)min(row + r * row_step, rows - 1) * stride;
#pragma unroll
      for (int i = 0; i < kUnit<FMT>; ++i) v[r][i] = 0;
#pragma unroll
      for (int k = 0; k < kBytes; ++k)
        if (k < blocks * kUnit<FMT>) v[r][k / 4] |= (uint32_t)at[k] << (8 * (k % 4));
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int i = 0; i < kUnit<FMT>; ++i) out[(row + r * row_step) * out_stride + i] = v[r][i];
}

// ---- up to 16 tokens: 16 NT rows of W per workgroup, whose waves take steps of
// 128 k in turn (together whole lines of every row) and add their sums through
// LDS at the end.  W and x of the next step are in flight while one is
// computed; x goes through LDS, where each wave keeps the rows of its step.
//
// Bound by the stream of W.  Reading nothing but W in this pattern takes 7.0 us
// for K4096 N16384 (10.3 for K7168) from the memory-side cache, 8.2 (12.6) from
// HBM; one MXFP4 token takes 8.6 and 12.8, 9.7 from HBM.  What was found on the
// way: fragments of x straight from memory cost as much as W itself (one token
// 13.4 us, 16 tokens 24), scales read step by step 3 us of 19.7 (a line each for
// 4 bytes), steps in runs per wave 1 to 2 us (the lines of the scales), streaming
// loads of W 2 to 6 us (inputs in the memory-side cache), three stages in
// flight nothing.
//
// DIAG (NVFP4, 4 XR tokens): a lane keeps its 16 bytes of W, 32 consecutive k of
// one row, two blocks.  x stands in the other operand so that rows 4 i .. 4 i + 3
// (one per token) hold the k's of lane row i and zeros elsewhere: the lanes of
// lane row i then get the products of their own weights alone, a block's sum
// per token, and multiply it by their own block's scale -- the weights go into
// the MFMA without it, one conversion for two of them instead of four instructions
// (one token, N16384: 9.5 us against 11.4).  They go in 2^-8 times their value,
// and the scales come with 2^8: 16 products of up to 6 x stay finite where x is,
// and every product is a multiple of 2^-142, which the sums hold.
// Else (16 tokens, of which 4 XR are staged): lane rows exchange dwords so that
// an MFMA takes 32 consecutive k, and the weights are scaled before it.
constexpr int kFewWaves = 8;
constexpr int kFewSeg = 128;  // steps whose scales are in LDS at a time

// Step units of a row's scales in LDS: an odd number, so that 16 rows lie in
// different banks.
__host__ __device__ inline int few_pitch(int steps) { return (steps < kFewSeg ? steps : kFewSeg) | 1; }

// 16-byte chunks of LDS in front of the scales: each wave's x, whose place its
// sums take, and four chunks of zeros.
template <bool DIAG, int XR, int NT>
constexpr int kFewShared = kFewWaves * 64 * std::max(XR, (DIAG ? XR : 1) * NT) + 4;

template <int FMT, bool DIAG, int XR, int NT, int OCC>
__global__ __launch_bounds__(64 * kFewWaves, OCC) void matvec_few_kernel(MatvecParams p) {
  static_assert(!DIAG || FMT == kNvfp4, "");
  constexpr int kBlock = FMT == kNvfp4 ? 16 : 32, kRows = 4 * XR, T = DIAG ? XR : 1;
  constexpr int kX = kRows * 16, kZeros = kFewShared<DIAG, XR, NT> - 4;
  extern __shared__ u32x4 lds[];
  uint32_t* scales = reinterpret_cast<uint32_t*>(lds + kZeros + 4);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15,
            part = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
  const int rows = (int)min((int64_t)(16 * NT), p.N - n0), tokens = (int)p.M;
  // uniform bases and 32-bit offsets of the lane
  const uint8_t* wq = p.w_q + n0 * (p.K / 2);
  const uint8_t* ws = p.w_s + n0 * (p.K / kBlock);
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(p.x);
  uint32_t wo[NT], xo[XR];
#pragma unroll
  for (int u = 0; u < NT; ++u) wo[u] = (uint32_t)min(16 * u + col, rows - 1) * (uint32_t)(p.K / 2) + 16 * part;
#pragma unroll
  for (int i = 0; i < XR; ++i) xo[i] = (uint32_t)min(4 * i + part, tokens - 1) * (uint32_t)(2 * p.K) + 16 * col;
  const int steps = (p.K + kMvStep - 1) / kMvStep, full = p.K / kMvStep, rest = (p.K - full * kMvStep) / 32;
  const int pitch = few_pitch(steps) * kUnit<FMT>;
  // x: row r's chunk q of a step sits at q ^ (r % 16), so that the 16 rows that
  // a fragment read covers, and the 16 chunks that a write covers, lie in
  // different banks
  u32x4* xl = lds + wave * kX;
  const bool diag = (col >> 2) == part;
  // DIAG: chunk 4 part + j of token col % 4 is at chunk `at` ^ j, or there are zeros
  const int at = diag ? wave * kX + (col & 3) * 16 + ((4 * part) ^ (col & 3)) : kZeros;
  if (DIAG && tid < 4) lds[kZeros + tid] = u32x4{0, 0, 0, 0};
  f32x4 acc[T][NT];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int u = 0; u < NT; ++u) acc[t][u] = f32x4{0, 0, 0, 0};

  struct Stage {
    u32x4 w[NT], x[XR];
  };
  auto load = [&](Stage& g, int c) {
    const uint8_t *q = wq + (size_t)c * (kMvStep / 2), *x = xb + (size_t)c * (2 * kMvStep);
#pragma unroll
    for (int u = 0; u < NT; ++u) g.w[u] = *reinterpret_cast<const u32x4*>(q + wo[u]);
#pragma unroll
    for (int i = 0; i < XR; ++i) g.x[i] = *reinterpret_cast<const u32x4*>(x + xo[i]);
  };
  auto compute = [&](const Stage& g, int step) {  // step: of the segment
    wave_sync();
#pragma unroll
    for (int i = 0; i < XR; ++i) xl[(4 * i + part) * 16 + (col ^ ((4 * i + part) & 15))] = g.x[i];
    wave_sync();
    if constexpr (DIAG) {
      u32x4 a[XR][4];
#pragma unroll
      for (int t = 0; t < XR; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) a[t][j] = lds[(t && diag ? (at ^ (4 * t)) + 64 * t : at) ^ j];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        // the lane's two scales are 16 bits of the row's 8 bytes
        const uint32_t s = reinterpret_cast<const uint16_t*>(scales + (16 * u + col) * pitch + step * 2)[part];
        const auto sc = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(s, 256.0f, false);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bf16x8 b0 = weights8<kMxfp4>(g.w[u][2 * h], 0x1p-8f), b1 = weights8<kMxfp4>(g.w[u][2 * h + 1], 0x1p-8f);
#pragma unroll
          for (int t = 0; t < XR; ++t) {
            const f32x4 v = mfma16(a[t][2 * h + 1], b1, mfma16(a[t][2 * h], b0, f32x4{0, 0, 0, 0}));
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][u][r] = __builtin_fmaf(v[r], sc[h], acc[t][u][r]);
          }
        }
      }
    } else {
      u32x4 w[NT];
      uint32_t s[NT][kUnit<FMT>];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        w[u] = exchange(g.w[u]);
#pragma unroll
        for (int i = 0; i < kUnit<FMT>; ++i) {
          s[u][i] = scales[(16 * u + col) * pitch + step * kUnit<FMT> + i];
          if constexpr (FMT == kNvfp4) s[u][i] >>= 8 * (part >> 1);
        }
      }
      const int r = min(col, kRows - 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // 32 k: one MFMA, its lane row `part` the k's 8 part .. 8 part + 8
        const u32x4 a = xl[r * 16 + ((4 * j + part) ^ r)];
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          float sc;
          if constexpr (FMT == kNvfp4) sc = j & 1 ? __builtin_amdgcn_cvt_f32_fp8(s[u][j / 2], 2)
                                                  : __builtin_amdgcn_cvt_f32_fp8(s[u][j / 2], 0);
          else sc = __uint_as_float(((s[u][0] >> (8 * j)) & 0xff) << 23);
          acc[0][u] = mfma16(a, weights8<FMT>(w[u][j], sc), acc[0][u]);
        }
      }
    }
  };

  for (int seg = 0; seg < steps; seg += kFewSeg) {
    const int end = min(seg + kFewSeg, full), held = min(seg + kFewSeg, steps) - seg;
    Stage even, odd;
    int c = seg + wave;
    if (c < end) load(even, c);
    // the scales of the segment: a wave takes rows in turn, its lanes the steps
    if (seg) __syncthreads();
    for (int i = lane; i < held; i += 64)
      stage_step<FMT, 16 * NT / kFewWaves>(ws + (size_t)(seg + i) * (kMvStep / kBlock), wave, kFewWaves, rows,
                                           p.K / kBlock, seg + i < full ? 4 : rest, scales + i * kUnit<FMT>, pitch);
    __syncthreads();
    // two steps a turn, each computed while the next is on its way
    for (; c + 2 * kFewWaves < end; c += 2 * kFewWaves) {
      load(odd, c + kFewWaves);
      compute(even, c - seg);
      load(even, c + 2 * kFewWaves);
      compute(odd, c + kFewWaves - seg);
    }
    if (c + kFewWaves < end) {
      load(odd, c + kFewWaves);
      compute(even, c - seg);
      compute(odd, c + kFewWaves - seg);
    } else if (c < end) {
      compute(even, c - seg);
    }
    if (rest && full < seg + kFewSeg && (full - seg) % kFewWaves == wave) {  // the partial step, zeros behind the row's end
      const uint8_t *q = wq + (size_t)full * (kMvStep / 2), *x = xb + (size_t)full * (2 * kMvStep);
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        even.w[u] = u32x4{0, 0, 0, 0};
        if (part < rest) even.w[u] = *reinterpret_cast<const u32x4*>(q + wo[u]);
      }
#pragma unroll
      for (int i = 0; i < XR; ++i) {
        even.x[i] = u32x4{0, 0, 0, 0};
        if (col < 4 * rest) even.x[i] = *reinterpret_cast<const u32x4*>(x + xo[i]);
      }
      compute(even, full - seg);
    }
  }

  const float scale = FMT == kNvfp4 ? p.w_gs[0] : 1.0f;
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int u = 0; u < NT; ++u) red[((wave * T + t) * NT + u) * 64 + lane] = acc[t][u];
  __syncthreads();
  if constexpr (DIAG) {
    const float* sums = reinterpret_cast<const float*>(lds);
    for (int i = tid; i < T * NT * 64; i += 64 * kFewWaves) {  // four tokens, row tile, row, token
      const int tu = i >> 6, e = i & 63;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w)
#pragma unroll
        for (int q = 0; q < 4; ++q) v += sums[((w * T * NT + tu) * 64 + 16 * q) * 4 + e];
      store_result(p, 4 * (tu / NT) + (e & 3), n0 + 16 * (tu % NT) + (e >> 2), v * scale);
    }
  } else {
    for (int i = tid; i < NT * 64; i += 64 * kFewWaves) {
      f32x4 v = red[i];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) v += red[w * NT * 64 + i];
#pragma unroll
      for (int r = 0; r < 4; ++r) store_result(p, 4 * ((i >> 4) & 3) + r, n0 + 16 * (i >> 6) + (i & 15), v[r] * scale);
    }
  }
}

// ---- up to 64 tokens per slice: ROWS rows of W per workgroup and the tokens in
// MT tiles of 16, both operands streamed into LDS in chunks of 256 k, two
// chunks ahead, and read from there by the wave that needs them: the waves
// share the rows by 32 (or 16) and a chunk's eight blocks of 32 k.
//
// Bound by the streams into LDS and by what a CU does with them, each by itself
// nearly as long as both (M64 K4096 N16384: 16.5 us NVFP4, 13.7 MXFP4; the loads
// alone 13.1 and 12.4, everything but the loads 14.2 and 11.4): 32 KiB of x and 8
// of W per chunk and CU; a conversion and two multiplications per pair of NVFP4
// weights beside the MFMAs, which share the issue slots of a SIMD; the fragments'
// way out of LDS, a barrier.  64 rows with two waves per SIMD instead of four:
// 18.0 and 13.6.  Measured and not kept: fragments read a chunk ahead (NVFP4 16.4,
// MXFP4 13.8 and more for fewer rows); conversions spread between the MFMAs by
// hand, x and W loaded by different waves with W four chunks ahead, chunks in
// another order per workgroup (0 to 15 % slower).
constexpr int kTileK = 256, kTileStages = 3;
constexpr int kTileSeg = 32;  // chunks whose scales are in LDS at a time

template <int FMT, int MT, int ROWS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES / 4) void matvec_tile_kernel(MatvecParams p) {
  constexpr int kBlock = FMT == kNvfp4 ? 16 : 32;
  constexpr int U = ROWS >= 32 ? 2 : 1, RG = ROWS / (16 * U), KS = WAVES / RG, JB = 8 / KS;  // row tiles of a wave, row groups, shares of k, blocks of one
  constexpr int kXChunks = 16 * MT * 32, kStage = kXChunks + ROWS * 8;  // 16-byte chunks
  extern __shared__ u32x4 lds[];
  uint32_t* scales = reinterpret_cast<uint32_t*>(lds + kTileStages * kStage);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15,
            part = lane >> 4, rg = wave % RG, ks = wave / RG;
  const int64_t n0 = (int64_t)blockIdx.x * ROWS, m0 = (int64_t)blockIdx.y * (16 * MT);
  const int rows = (int)min((int64_t)ROWS, p.N - n0), tokens = (int)min((int64_t)(16 * MT), p.M - m0);
  const uint8_t* wq = p.w_q + n0 * (p.K / 2);
  const uint8_t* ws = p.w_s + n0 * (p.K / kBlock);
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(p.x + m0 * p.K);
  const int chunks = (p.K + kTileK - 1) / kTileK;

  // This lane's sources.  A stage is filled a KiB per load, wave w loads w, w +
  // WAVES ..: first token rows two at a time, 32 pieces of 8 k each, token row r's
  // piece q at q ^ (r % 16); then W's rows eight at a time, 8 pieces of 32 k
  // each, in the order 0 8 1 9 .. of their 16, row n's piece q at q ^ (n % 8).
  // Rows in that order and places: every fragment read spreads over all banks.
  // Waves below ROWS / 8 load W too, and one of x more where WAVES does not
  // divide 8 MT.
  constexpr int kMostX = (8 * MT + WAVES - 1) / WAVES, kLeastX = 8 * MT / WAVES;
  static_assert(8 * MT % WAVES == 0 || 8 * MT % WAVES == ROWS / 8, "");
  uint32_t xo[kMostX];
#pragma unroll
  for (int k = 0; k < kMostX; ++k) {
    const int r = 2 * (wave + k * WAVES) + (lane >> 5);
    xo[k] = (uint32_t)min(r, tokens - 1) * (uint32_t)(2 * p.K) + 16 * ((lane & 31) ^ (r & 15));
  }
  const int slot = 8 * (wave & 1) + (lane >> 3), row = 16 * (wave >> 1) + (slot >> 1) + 8 * (slot & 1);
  const uint32_t wo = (uint32_t)min(row, rows - 1) * (uint32_t)(p.K / 2) + 16 * ((lane & 7) ^ (row & 7));
  const int full = p.K / kTileK;
  auto issue = [&](auto both, int c, int stage) {  // a whole chunk
    u32x4* st = lds + stage * kStage + 64 * wave;
#pragma unroll
    for (int k = 0; k < (both ? kMostX : kLeastX); ++k)
      dma16s(reinterpret_cast<f16x8*>(st + 64 * k * WAVES), xb + (size_t)c * (2 * kTileK), xo[k]);
    if constexpr (both) dma16s(reinterpret_cast<f16x8*>(st + kXChunks), wq + (size_t)c * (kTileK / 2), wo);
  };
  auto issue_any = [&](auto both, int c, int stage) {
    if (c < full) {
      issue(both, c, stage);
      return;
    }
    // pieces behind the row's end: the row's first one instead, their products
    // are left out.  (An offset holds 16 times its piece: never negative.)
    u32x4* st = lds + stage * kStage + 64 * wave;
    const uint32_t left = (uint32_t)(p.K - c * kTileK);
#pragma unroll
    for (int k = 0; k < (both ? kMostX : kLeastX); ++k) {
      const uint32_t piece = (lane & 31) ^ ((2 * (wave + k * WAVES) + (lane >> 5)) & 15);
      dma16s(reinterpret_cast<f16x8*>(st + 64 * k * WAVES), xb,
             8 * piece < left ? xo[k] + (uint32_t)c * (2 * kTileK) : xo[k] - 16 * piece);
    }
    const uint32_t piece = (lane & 7) ^ (row & 7);
    if constexpr (both)
      dma16s(reinterpret_cast<f16x8*>(st + kXChunks), wq,
             32 * piece < left ? wo + (uint32_t)c * (kTileK / 2) : wo - 16 * piece);
  };
  // the scales of chunks seg .. seg + kTileSeg: a wave takes rows in turn, its
  // lanes the steps of 128 k
  const int total = (p.K + kMvStep - 1) / kMvStep, whole = p.K / kMvStep, rest = (p.K - whole * kMvStep) / 32;
  const int pitch = (min(total, 2 * kTileSeg) | 1) * kUnit<FMT>;
  auto stage_scales = [&](int seg) {
    const int i = 2 * seg + lane;
    if (i < total)
      stage_step<FMT, ROWS / WAVES>(ws + (size_t)i * (kMvStep / kBlock), wave, WAVES, rows, p.K / kBlock,
                                         i < whole ? 4 : rest, scales + lane * kUnit<FMT>, pitch);
  };

  f32x4 acc[MT][U];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < U; ++u) acc[t][u] = f32x4{0, 0, 0, 0};
  // fragments of block b of a chunk: x piece 4 b + part of token row 16 t + col;
  // the dword of row 16 (U rg + u) + col with its 8 weights from 32 b + 8 part.
  // Byte offsets in a stage, and of the row's scales.
  const uint8_t* bytes = reinterpret_cast<const uint8_t*>(lds);
  int ao[JB], wd[JB], so[U];
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const int b = JB * ks + j;
    ao[j] = 16 * (col * 32 + ((4 * b + part) ^ col));
    wd[j] = 16 * (kXChunks + (16 * U * rg + 2 * (col & 7) + (col >> 3)) * 8 + (b ^ (col & 7))) + 4 * part;
  }
#pragma unroll
  for (int u = 0; u < U; ++u)  // block b's scales are bytes 2 b and 2 b + 1, or byte b
    so[u] = 16 * kTileStages * kStage + (16 * (U * rg + u) + col) * pitch * 4 +
            (FMT == kNvfp4 ? 2 * JB * ks + (part >> 1) : JB * ks);
  u32x4 a[JB][MT];
  uint32_t q[JB][U], sc[JB][U];
  auto read = [&](int c, int stage) {  // blocks behind the row's end hold something, and are not used
    const uint8_t* st = bytes + stage * (16 * kStage);
    const uint8_t* sp = bytes + (c % kTileSeg) * (8 * kUnit<FMT>);
#pragma unroll
    for (int j = 0; j < JB; ++j) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        q[j][u] = *reinterpret_cast<const uint32_t*>(st + wd[j] + u * (16 * 16 * 8));
        sc[j][u] = sp[so[u] + (FMT == kNvfp4 ? 2 : 1) * j];
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) a[j][t] = *reinterpret_cast<const u32x4*>(st + ao[j] + t * (16 * 16 * 32));
    }
  };
  auto compute = [&](auto whole, int blocks) {  // the chunk's number of blocks
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      if (!whole && JB * ks + j >= blocks) break;  // wave-uniform
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float s = FMT == kNvfp4 ? __builtin_amdgcn_cvt_f32_fp8(sc[j][u], 0) : __uint_as_float(sc[j][u] << 23);
        const bf16x8 v = weights8<FMT>(q[j][u], s);
#pragma unroll
        for (int t = 0; t < MT; ++t)
          acc[t][u] = mfma16(a[j][t], v, acc[t][u]);
      }
    }
  };

  // A copy of the loop for each of the two counts of loads, without a branch but
  // its own: the checks of one loop for all took 2 us of 19 (64 tokens, N16384).
  auto run = [&](auto both) {
    constexpr int kLoads = both ? kMostX + 1 : kLeastX;  // of this wave and a chunk
    issue_any(both, 0, 0);
    if (chunks > 1) issue_any(both, 1, 1);
    stage_scales(0);
    int c = 0, stage = 0;
    auto next = [&] {
      ++c;
      stage = stage == kTileStages - 1 ? 0 : stage + 1;
    };
    auto behind = [&] { return stage ? stage - 1 : kTileStages - 1; };  // chunk c + 2's stage, as c - 1's
    for (int seg = 0; c + 2 < full; seg += kTileSeg) {
      const int end = min(seg + kTileSeg, full - 2);
      if (seg) {
        lds_barrier();  // every wave has read the scales of chunk c - 1
        stage_scales(seg);
      }
#pragma unroll 1
      while (c < end) {
        wait_vmcnt<kLoads>();  // chunk c has landed, c + 1 may be on its way
        lds_barrier();         // for every wave, and every wave has read chunk c - 1
        read(c, stage);
        issue(both, c + 2, behind());
        SCHED_FENCE();  // the loads go out before the reads are waited for
        compute(std::true_type(), 8);
        next();
      }
    }
    while (c < chunks) {  // the same with every check, three chunks at most
      if (c + 1 < chunks) wait_vmcnt<kLoads>();
      else wait_vmcnt<0>();
      lds_barrier();
      if (c && c % kTileSeg == 0) {
        stage_scales(c);
        lds_barrier();
      }
      read(c, stage);
      if (c + 2 < chunks) issue_any(both, c + 2, behind());
      compute(std::false_type(), (p.K - c * kTileK) / 32);
      next();
    }
  };
  if (ROWS / 8 == WAVES || wave < ROWS / 8) run(std::true_type());
  else run(std::false_type());

  // the waves of a row group add their sums
  constexpr int kTiles = ROWS / 16, kSums = MT * kTiles * 64;
  const float scale = FMT == kNvfp4 ? p.w_gs[0] : 1.0f;
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < U; ++u) red[((ks * MT + t) * kTiles + U * rg + u) * 64 + lane] = acc[t][u];
  __syncthreads();
#pragma unroll
  for (int h = 0; h < (kSums + 64 * WAVES - 1) / (64 * WAVES); ++h) {
    const int i = tid + h * 64 * WAVES;
    if (i >= kSums) break;
    f32x4 v = red[i];
#pragma unroll
    for (int w = 1; w < KS; ++w) v += red[w * kSums + i];
    const int64_t n = n0 + 16 * ((i >> 6) % kTiles) + (i & 15), m = m0 + 16 * (i / (64 * kTiles)) + 4 * ((i >> 4) & 3);
#pragma unroll
    for (int r = 0; r < 4; ++r) store_result(p, m + r, n, v[r] * scale);
  }
}

template <int FMT, int MT, int ROWS, int WAVES>
void launch_tile(const MatvecParams& p, hipStream_t s) {
  const dim3 g((unsigned)((p.N + ROWS - 1) / ROWS), (unsigned)((p.M + 16 * MT - 1) / (16 * MT)));
  const int total = (p.K + kMvStep - 1) / kMvStep;
  constexpr int kStages = kTileStages * (16 * MT * 32 + ROWS * 8), kSums = WAVES / (ROWS > 32 ? 2 : 1) * MT * ROWS * 4;
  const size_t scales = 4 * (size_t)ROWS * (std::min(total, 2 * kTileSeg) | 1) * kUnit<FMT>;
  const size_t lds = std::max(16 * (size_t)kStages + scales, 16 * (size_t)kSums);  // the sums take the others' place
  matvec_tile_kernel<FMT, MT, ROWS, WAVES><<<g, 64 * WAVES, lds, s>>>(p);
}

// Workgroups that the device runs at once, one per CU.
constexpr int64_t kCus = 256;

// The smallest tile with which every workgroup has a CU of its own: all of them
// read all of x, so more than one on a CU costs what a larger tile saves, and
// with fewer rows a workgroup is done sooner (NVFP4 M64 K4096: N4096 10.2, 11.3 and
// 14.4 us with 16, 32 and 64 rows, N8192 18.2, 12.0 and 14.9, N16384 32.8, 21.6
// and 16.5; M32, of which two fit on a CU: N8192 10.3 with 16 rows and 9.2 with
// 32, N16384 14.6 with 32 and 12.4 with 64).  Beyond N16384 there is a second
// round, a mostly empty one at first (M64 K4096: N18432 28.0 us, N28672 29.3; MXFP4
// 23.9 and 25.2).
template <int FMT, int MT>
void launch_tiles(const MatvecParams& p, hipStream_t s) {
  const int64_t slices = (p.M + 16 * MT - 1) / (16 * MT);
  if ((p.N + 15) / 16 * slices <= kCus) launch_tile<FMT, MT, 16, 8>(p, s);
  else if ((p.N + 31) / 32 * slices <= kCus) launch_tile<FMT, MT, 32, 8>(p, s);
  else launch_tile<FMT, MT, 64, 16>(p, s);
}

template <int FMT, bool DIAG, int XR, int NT, int OCC>
void launch_few(const MatvecParams& p, hipStream_t s) {
  const size_t lds = 16 * (size_t)kFewShared<DIAG, XR, NT> +
                     4 * (size_t)(16 * NT) * few_pitch((p.K + kMvStep - 1) / kMvStep) * kUnit<FMT>;
  matvec_few_kernel<FMT, DIAG, XR, NT, OCC>
      <<<(unsigned)((p.N + 16 * NT - 1) / (16 * NT)), 64 * kFewWaves, lds, s>>>(p);
}

// Which kernel, by what was measured on both sides (us, K4096 unless it says).
//   M <= 4: a few rows per workgroup, 16, or for NVFP4 32 where workgroups of 32
//   run at once and those of 16 do not, three of which fit on a CU (M1: N16384
//   9.1 against 10.8, N12288 8.6 against 7.8, N18432 12.4 against 11.6).  MXFP4
//   with many rows takes the tiles (M4 K7168 N28672 21.9 against 27.3; NVFP4 never).
//   M <= 8: 16 rows up to three workgroups per CU, for NVFP4 64 where these run
//   at once and three of 16 do not (K7168: N16384 15.4 against 16.1 with the
//   tiles, N20480 20.7 with the tiles against 21.8; MXFP4 N12288 11.0 against
//   12.4, N14336 13.9 against 12.5).
//   M <= 16: 16 rows up to two per CU.  N4096 is clear (6.1 against 8.0 with the
//   tiles, MXFP4 5.2 against 6.7), and so is N10240 (11.2 against 10.9, MXFP4 10.1
//   against 9.0).  Between, with W from HBM, where a decode step finds it, N8192:
//   NVFP4 M9 9.3 against 9.7, M16 10.1 against 9.9; MXFP4 8.3 against 9.0 and 9.4
//   against 9.2; K7168 NVFP4 13.2 against 14.1 and 15.2 against 14.2, MXFP4 12.4
//   against 13.2 and 14.4 against 13.4; K2048 6.8 against 6.8 and 7.3 against 6.9,
//   MXFP4 5.9 against 6.2 and 6.5 against 6.3.  With W in the memory-side cache
//   the tiles are ahead by 1 to 2 %, MXFP4 by 2 to 9 %.
//   The tiles of up to 16 tokens: 32 rows where three per CU hold all of them
//   (K7168: NVFP4 N24576 25.7 against 33.1 with 64 rows, N28672 36.3 against 28.9).
template <int FMT>
void launch_format(const MatvecParams& p, hipStream_t s) {
  const int64_t rows16 = (p.N + 15) / 16, rows32 = (p.N + 31) / 32, rows64 = (p.N + 63) / 64;
  const bool at_once = rows16 <= 3 * kCus;  // 16-row workgroups run all at once
  if (p.M <= 4 && (FMT == kNvfp4 || rows16 <= 7 * kCus)) {
    if constexpr (FMT == kMxfp4) launch_few<FMT, false, 1, 1, 8>(p, s);
    else if (!at_once && rows32 <= 2 * kCus) launch_few<FMT, true, 1, 2, 4>(p, s);
    else launch_few<FMT, true, 1, 1, 6>(p, s);
  } else if (p.M <= 8 && (at_once || (FMT == kNvfp4 && rows64 <= kCus))) {
    if constexpr (FMT == kMxfp4) launch_few<FMT, false, 2, 1, 6>(p, s);
    else if (at_once) launch_few<FMT, true, 2, 1, 4>(p, s);
    else launch_few<FMT, true, 2, 4, 2>(p, s);
  } else if (p.M <= 16 && rows16 <= 2 * kCus) {
    launch_few<FMT, false, 4, 1, 4>(p, s);
  } else if (p.M <= 16) {
    if (rows32 <= 3 * kCus) launch_tile<FMT, 1, 32, 8>(p, s);
    else launch_tile<FMT, 1, 64, 8>(p, s);
  } else if (p.M <= 32) {
    launch_tiles<FMT, 2>(p, s);
  } else if (p.M <= 48) {
    launch_tiles<FMT, 3>(p, s);
  } else {
    launch_tiles<FMT, 4>(p, s);
  }
}

}  // namespace

hipError_t launch_matvec(int fmt, const uint16_t* x, int64_t M, int K, const uint8_t* w_q, const uint8_t* w_s,
                         const float* w_gs, int64_t N, bool bf16_out, void* out, hipStream_t s) {
  if (M == 0) return hipSuccess;
  const MatvecParams p = {x, w_q, w_s, w_gs, out, M, N, K, bf16_out};
  if (fmt == kNvfp4) launch_format<kNvfp4>(p, s);
  else launch_format<kMxfp4>(p, s);
  return hipGetLastError();
}

}  // namespace nvfp4
