// Products of a few tokens with 4-bit weights on gfx950: y[m][n] = gs * sum_k
// x[m][k] * e2m1(w[n][k]) * scale[n][k / g], x bf16, W NVFP4 (E4M3 scale per 16,
// fp32 tensor scale) or MXFP4 (E8M0 scale per 32).
//
// e2m1 * scale has at most 6 significant bits for E4M3 and 2 for E8M0, so every
// weight is a bf16 value exactly, every product is exact and the matrix cores
// accumulate in fp32; the tensor scale multiplies the sum.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "launch.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct MatvecParams {
  const uint16_t* x;    // bf16 [M][K]
  const uint8_t* w_q;   // [N][K/2]
  const uint8_t* w_s;   // [N][K/16] or [N][K/32]
  const float* w_gs;    // NVFP4 only
  void* out;            // [M][N]
  int64_t M, N;
  int K;
};

constexpr int kMvWaves = 8;
constexpr int kMvStep = 128;  // K per wave and step: a lane's 32 weights are 16 bytes

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

// 16 rows of W per workgroup, MT * 16 tokens; the waves take steps of K in
// turn and their sums are added through LDS.
template <int FMT, int MT, bool BF16_OUT>
__global__ __launch_bounds__(64 * kMvWaves) void matvec_kernel(MatvecParams p) {
  __shared__ f32x4 red[kMvWaves][MT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, part = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT);
  const int64_t n = min(n0 + col, p.N - 1);
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4{0, 0, 0, 0};
  for (int k0 = wave * kMvStep; k0 < p.K; k0 += kMvWaves * kMvStep) {
    const int k = k0 + 32 * part;
    const bool on = k < p.K;
    const int kk = on ? k : 0;
    uint4 w = *reinterpret_cast<const uint4*>(p.w_q + n * (p.K / 2) + kk / 2);
    if (!on) w = make_uint4(0, 0, 0, 0);
    float s0, s1;
    if constexpr (FMT == kMxfp4) {
      s0 = s1 = __uint_as_float((uint32_t)p.w_s[n * (p.K / 32) + kk / 32] << 23);
    } else {
      const uint32_t s = *reinterpret_cast<const uint16_t*>(p.w_s + n * (p.K / 16) + kk / 16);
      s0 = e4m3_decode_signed(s & 0xff);
      s1 = e4m3_decode_signed(s >> 8);
    }
    const bf16x8 b[4] = {weights8<FMT>(w.x, s0), weights8<FMT>(w.y, s0), weights8<FMT>(w.z, s1),
                         weights8<FMT>(w.w, s1)};
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint4* x = reinterpret_cast<const uint4*>(p.x + min(m0 + 16 * t + col, p.M - 1) * p.K + kk);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 a = x[j];
        if (!on) a = make_uint4(0, 0, 0, 0);
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), b[j], acc[t], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) red[wave][t][lane] = acc[t];
  __syncthreads();
  const float g = FMT == kNvfp4 ? p.w_gs[0] : 1.0f;
  for (int i = tid; i < MT * 64; i += 64 * kMvWaves) {
    f32x4 s = red[0][i >> 6][i & 63];
    for (int w = 1; w < kMvWaves; ++w) s += red[w][i >> 6][i & 63];
    const int64_t nn = n0 + (i & 15);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t m = m0 + 16 * (i >> 6) + 4 * ((i >> 4) & 3) + r;
      if (m < p.M && nn < p.N) {
        const float v = s[r] * g;
        if constexpr (BF16_OUT) static_cast<__bf16*>(p.out)[m * p.N + nn] = (__bf16)v;
        else static_cast<float*>(p.out)[m * p.N + nn] = v;
      }
    }
  }
}

template <int FMT, int MT>
void launch_as(const MatvecParams& p, bool bf16_out, hipStream_t s) {
  const dim3 g((unsigned)((p.N + 15) / 16), (unsigned)((p.M + 16 * MT - 1) / (16 * MT)));
  if (bf16_out) matvec_kernel<FMT, MT, true><<<g, 64 * kMvWaves, 0, s>>>(p);
  else matvec_kernel<FMT, MT, false><<<g, 64 * kMvWaves, 0, s>>>(p);
}

template <int FMT>
void launch_format(const MatvecParams& p, bool bf16_out, hipStream_t s) {
  if (p.M <= 16) launch_as<FMT, 1>(p, bf16_out, s);
  else if (p.M <= 32) launch_as<FMT, 2>(p, bf16_out, s);
  else launch_as<FMT, 4>(p, bf16_out, s);
}

}  // namespace

hipError_t launch_matvec(int fmt, const uint16_t* x, int64_t M, int K, const uint8_t* w_q, const uint8_t* w_s,
                         const float* w_gs, int64_t N, bool bf16_out, void* out, hipStream_t s) {
  if (M == 0) return hipSuccess;
  const MatvecParams p = {x, w_q, w_s, w_gs, out, M, N, K};
  if (fmt == kNvfp4) launch_format<kNvfp4>(p, bf16_out, s);
  else launch_format<kMxfp4>(p, bf16_out, s);
  return hipGetLastError();
}

}  // namespace nvfp4
