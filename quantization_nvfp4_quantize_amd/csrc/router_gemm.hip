// The router's gate projection on gfx950: logits[t][e] = sum_k x[t][k] w[e][k]
// (+ bias[e]), x bf16, w bf16 or fp32, logits fp32.
//
// Products are exact and accumulated in fp32 on the matrix cores.  A 24-bit
// fp32 weight is the sum of three bf16 values (its bits taken eight at a
// time), so an fp32 weight costs three products of which each is exact; a
// single rounding of w to bf16 would move the logits by 2^-9 of their terms
// and with them the choice of experts.
#include <hip/hip_runtime.h>

#include "launch.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct GateParams {
  const uint16_t* x;  // bf16 [T][H]
  const void* w;      // bf16 or fp32 [E][H]
  const float* bias;  // nullable [E]
  float* out;         // [T][E]
  int64_t T;
  int H, E;
};

__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

// Eight fp32 values as three bf16 fragments whose sum is exact: each takes
// the upper half of what is left.
struct Split3 {
  uint4 f[3];
};
__device__ __forceinline__ Split3 split3(const float4& a, const float4& b) {
  float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t d[3][4];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = __float_as_uint(v[2 * i]), hi = __float_as_uint(v[2 * i + 1]);
      d[p][i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
      v[2 * i] -= __uint_as_float(lo & 0xffff0000u);
      v[2 * i + 1] -= __uint_as_float(hi & 0xffff0000u);
    }
  }
  Split3 s;
#pragma unroll
  for (int p = 0; p < 3; ++p) s.f[p] = make_uint4(d[p][0], d[p][1], d[p][2], d[p][3]);
  return s;
}

// ---- few tokens: one workgroup computes 16 tokens x 16 experts, its waves a
// slice of K each.  Every wave has 8 K steps of both operands (64 registers
// of loads) in flight, which is what a call over 3.7 MB of weights needs: it
// lasts about as long as its longest chain of loads.
constexpr int kSmallWaves = 16;
constexpr int kSmallSteps = 8;

template <bool F32W>
__global__ __launch_bounds__(64 * kSmallWaves) void gate_small_kernel(GateParams p) {
  __shared__ float part[kSmallWaves][16 * 17];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int etiles = (p.E + 15) / 16;
  const int e0 = (int)(blockIdx.x % etiles) * 16;
  const int64_t t0 = (int64_t)(blockIdx.x / etiles) * 16;
  const int r = lane & 15, g = lane >> 4;
  const int64_t t = min(t0 + r, p.T - 1);
  const int e = min(e0 + r, p.E - 1);
  const uint16_t* xr = p.x + t * p.H + 8 * g;
  const int64_t wo = (int64_t)e * p.H + 8 * g;
  const int nk = p.H / 32;
  const int k0 = nk * wave / kSmallWaves, k1 = nk * (wave + 1) / kSmallWaves;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = k0; k < k1; k += kSmallSteps) {
    uint4 a[kSmallSteps];
    if constexpr (F32W) {
      float4 b[kSmallSteps][2];
#pragma unroll
      for (int i = 0; i < kSmallSteps; ++i) {
        const int kk = min(k + i, k1 - 1);
        a[i] = *reinterpret_cast<const uint4*>(xr + 32 * kk);
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + wo + 32 * kk);
        b[i][0] = s[0];
        b[i][1] = s[1];
      }
#pragma unroll
      for (int i = 0; i < kSmallSteps; ++i) {
        if (k + i < k1) {
          const Split3 s = split3(b[i][0], b[i][1]);
#pragma unroll
          for (int q = 2; q >= 0; --q) acc = mfma16(a[i], s.f[q], acc);
        }
      }
    } else {
      uint4 b[kSmallSteps];
#pragma unroll
      for (int i = 0; i < kSmallSteps; ++i) {
        const int kk = min(k + i, k1 - 1);
        a[i] = *reinterpret_cast<const uint4*>(xr + 32 * kk);
        b[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.w) + wo + 32 * kk);
      }
#pragma unroll
      for (int i = 0; i < kSmallSteps; ++i)
        if (k + i < k1) acc = mfma16(a[i], b[i], acc);
    }
  }
  // element i of the accumulator: token 4 (lane / 16) + i, expert lane % 16
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][17 * (4 * g + i) + r] = acc[i];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int tr = threadIdx.x >> 4, ec = threadIdx.x & 15;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) v += part[w][17 * tr + ec];
    if (t0 + tr < p.T && e0 + ec < p.E) p.out[(t0 + tr) * p.E + e0 + ec] = v + (p.bias ? p.bias[e0 + ec] : 0.0f);
  }
}

}  // namespace

size_t router_logits_workspace_bytes(int64_t T, int64_t H, int64_t E, bool w_bf16) {
  (void)T, (void)H, (void)E, (void)w_bf16;
  return 0;
}

hipError_t launch_router_logits(const uint16_t* x, int64_t T, int H, const void* w, bool w_bf16, int E,
                                const float* bias, float* out, void* ws, hipStream_t s) {
  (void)ws;
  GateParams p{x, w, bias, out, T, H, E};
  const int64_t tiles = (T + 15) / 16 * ((E + 15) / 16);
  const dim3 grid((unsigned)tiles), block(64 * kSmallWaves);
  if (w_bf16)
    gate_small_kernel<false><<<grid, block, 0, s>>>(p);
  else
    gate_small_kernel<true><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace nvfp4
