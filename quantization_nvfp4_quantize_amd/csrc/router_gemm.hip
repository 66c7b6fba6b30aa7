// The router's gate projection on gfx950: logits[t][e] = sum_k x[t][k] w[e][k]
// (+ bias[e]), x bf16, w bf16 or fp32, logits fp32.
//
// Products are exact and accumulated in fp32 on the matrix cores.  A 24-bit
// fp32 weight is the sum of three bf16 values (its bits taken eight at a
// time), so an fp32 weight costs three products of which each is exact; a
// single rounding of w to bf16 would move the logits by 2^-9 of their terms
// and with them the choice of experts.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gemm_common.hpp"
#include "launch.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct GateParams {
  const uint16_t* x;  // bf16 [T][H]
  const void* w;      // bf16 or fp32 [E][H]; the tiled kernel: bf16 planes [planes][E][H]
  const float* bias;  // nullable [E]
  float* out;         // [T][E], or the partial sums [parts][T][E]
  int64_t T;
  int H, E;
  int parts;          // partial sums per logit (1: out is the result, with the bias)
  int slices;         // slices of K
};

__device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

__device__ __forceinline__ void store_logit(const GateParams& p, int part, int64_t t, int e, float v) {
  if (t < p.T && e < p.E) p.out[((int64_t)part * p.T + t) * p.E + e] = p.parts == 1 && p.bias ? v + p.bias[e] : v;
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

// ---- one to four tokens: a workgroup per expert, every thread a few 16-byte
// chunks of the row, all of them requested at once: one launch that lasts one
// trip to memory.  fp32 fused multiply-adds keep the products exact.
constexpr int kDotThreads = 256;
constexpr int kDotTokens = 4;

template <bool F32W, int NT>
__global__ __launch_bounds__(kDotThreads) void gate_dot_kernel(GateParams p) {
  constexpr int kUnroll = 4;
  __shared__ float part[kDotThreads / 64][NT];
  const int e = blockIdx.x, tid = threadIdx.x, chunks = p.H / 8;
  float acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = 0.0f;
  for (int c0 = tid; c0 < chunks; c0 += kUnroll * kDotThreads) {
    uint4 xv[kUnroll][NT];
    float wv[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int c = c0 + u * kDotThreads;
      const int64_t at = (int64_t)e * p.H + 8 * (int64_t)min(c, chunks - 1);
      if constexpr (F32W) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + at);
        const float4 lo = s[0], hi = s[1];
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) wv[u][i] = v[i];
      } else {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.w) + at);
        const uint32_t d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          wv[u][2 * i] = bf16_lo(d[i]);
          wv[u][2 * i + 1] = bf16_hi(d[i]);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
        xv[u][t] = *reinterpret_cast<const uint4*>(p.x + min((int64_t)t, p.T - 1) * p.H +
                                                   8 * (int64_t)min(c, chunks - 1));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (c0 + u * kDotThreads < chunks) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t d[4] = {xv[u][t].x, xv[u][t].y, xv[u][t].z, xv[u][t].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[t] = __builtin_fmaf(bf16_lo(d[i]), wv[u][2 * i], acc[t]);
            acc[t] = __builtin_fmaf(bf16_hi(d[i]), wv[u][2 * i + 1], acc[t]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[t] += __shfl_xor(acc[t], o);
    if ((tid & 63) == 0) part[tid >> 6][t] = acc[t];
  }
  __syncthreads();
  if (tid < NT) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kDotThreads / 64; ++w) v += part[w][tid];
    store_logit(p, 0, tid, e, v);
  }
}

// ---- few tokens: 32 tokens x 32 experts and a slice of K per workgroup, a
// quarter of the slice per wave, operands straight from memory into
// registers.  A call of this size lasts about as long as its longest chain of
// loads, so the slices are short: a wave has its whole share in flight at once
// where K allows.  Workgroups that run on one XCD (blockIdx % 8) take the same
// slices, so an XCD's L2 fetches its part of x and w and not all of both.
constexpr int kSliceWaves = 4;
constexpr int kSliceTile = 32;

template <bool F32W>
__global__ __launch_bounds__(64 * kSliceWaves) void gate_slice_kernel(GateParams p) {
  constexpr int kSteps = F32W ? 8 : 16;  // K steps of 16 in flight
  __shared__ float part[kSliceWaves][32 * 33];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int etiles = (p.E + kSliceTile - 1) / kSliceTile;
  const int slice = blockIdx.x % p.slices, tile = blockIdx.x / p.slices;
  const int e0 = tile % etiles * kSliceTile;
  const int64_t t0 = (int64_t)(tile / etiles) * kSliceTile;
  const int r = lane & 31, g = lane >> 5;
  const uint16_t* xr = p.x + min(t0 + r, p.T - 1) * p.H + 8 * g;
  const int64_t wo = (int64_t)min(e0 + r, p.E - 1) * p.H + 8 * g;
  const int nk = p.H / 16, share = p.slices * kSliceWaves, mine = slice * kSliceWaves + wave;
  const int k0 = (int)((int64_t)nk * mine / share), k1 = (int)((int64_t)nk * (mine + 1) / share);
  f32x16 acc = {};
  for (int k = k0; k < k1; k += kSteps) {
    uint4 a[kSteps];
    if constexpr (F32W) {
      float4 b[kSteps][2];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int kk = 16 * min(k + i, k1 - 1);
        a[i] = *reinterpret_cast<const uint4*>(xr + kk);
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + wo + kk);
        b[i][0] = s[0];
        b[i][1] = s[1];
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (k + i < k1) {
          const Split3 s = split3(b[i][0], b[i][1]);
#pragma unroll
          for (int q = 2; q >= 0; --q) acc = mfma32(a[i], s.f[q], acc);
        }
      }
    } else {
      uint4 b[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int kk = 16 * min(k + i, k1 - 1);
        a[i] = *reinterpret_cast<const uint4*>(xr + kk);
        b[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.w) + wo + kk);
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (k + i < k1) acc = mfma32(a[i], b[i], acc);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) part[wave][33 * acc_row(i, lane) + r] = acc[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * 32; i += 64 * kSliceWaves) {
    const int row = i >> 5, col = i & 31;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kSliceWaves; ++w) v += part[w][33 * row + col];
    store_logit(p, slice, t0 + row, e0 + col, v);
  }
}

// ---- many tokens: 128 tokens x 128 experts per workgroup, 64 x 64 per wave
// (2 x 2 MFMA tiles of 32 x 32), K in steps of 64 through four LDS stages
// filled by direct loads three steps ahead.  Chunk c (16 bytes) of a row lies
// at c ^ swz_key(row).  With too few tiles for the chip, K is sliced as well;
// an fp32 weight comes as three bf16 planes (gate_planes_kernel), each a
// partial sum of its own.
constexpr int kTileRows = 128;
constexpr int kTileStages = 4;
constexpr int kTileOperand = kTileRows * 8;  // 16-byte chunks of one operand's stage

__global__ __launch_bounds__(256) void gate_tile_kernel(GateParams p) {
  __shared__ uint4 lds[kTileStages * 2 * kTileOperand];
  const int etiles = (p.E + kTileRows - 1) / kTileRows;
  const int ttiles = (int)((p.T + kTileRows - 1) / kTileRows);
  int item;
  if (!work_item(etiles * ttiles * p.parts, &item)) return;
  const int part = item / (etiles * ttiles), tile = item % (etiles * ttiles);
  const int slice = part % p.slices, plane = part / p.slices;
  const int e0 = tile % etiles * kTileRows;
  const int64_t t0 = (int64_t)(tile / etiles) * kTileRows;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = p.H / 64;
  const int s0 = (int)((int64_t)steps * slice / p.slices), s1 = (int)((int64_t)steps * (slice + 1) / p.slices);
  const uint32_t row_bytes = 2u * (uint32_t)p.H;
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(p.x) + t0 * row_bytes;
  const uint8_t* wb = static_cast<const uint8_t*>(p.w) + ((int64_t)plane * p.E + e0) * row_bytes;
  const int trows = (int)min((int64_t)kTileRows, p.T - t0), erows = min(kTileRows, p.E - e0);
  // load u of a wave: rows 32 wave + 8 u .. + 7 of each operand, 128 bytes each
  uint32_t xo[4], wo[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int row = 32 * wave + 8 * u + (lane >> 3);
    const uint32_t chunk = 16u * (uint32_t)((lane & 7) ^ swz_key(row));
    xo[u] = (uint32_t)min(row, trows - 1) * row_bytes + chunk;  // rows past the end repeat the last one
    wo[u] = (uint32_t)min(row, erows - 1) * row_bytes + chunk;
  }
  auto load = [&](int step, int stage) {
    uint4* dst = lds + stage * 2 * kTileOperand + 32 * 8 * wave;
    const size_t at = (size_t)step * 128;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      dma16s(reinterpret_cast<f16x8*>(dst + 64 * u), xb + at, xo[u]);
      dma16s(reinterpret_cast<f16x8*>(dst + kTileOperand + 64 * u), wb + at, wo[u]);
    }
  };
  const int wm = wave >> 1, wn = wave & 1, r = lane & 31, g = lane >> 5;
  const uint4 *fa[2], *fb[2];
  int ka[2], kb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int ra = 64 * wm + 32 * i + r, rb = 64 * wn + 32 * i + r;
    fa[i] = lds + 8 * ra;
    fb[i] = lds + kTileOperand + 8 * rb;
    ka[i] = swz_key(ra);
    kb[i] = swz_key(rb);
  }
  f32x16 acc[2][2] = {};
#pragma unroll
  for (int i = 0; i < kTileStages - 1; ++i) load(min(s0 + i, s1 - 1), i);
  for (int s = s0; s < s1; ++s) {
    const int stage = (s - s0) & (kTileStages - 1);
    // 8 loads a step: two later steps may still be on their way
    wait_vmcnt<16>();
    lds_barrier();  // stage s has landed for every wave, and stage s - 1 has been read by every wave
    load(min(s + kTileStages - 1, s1 - 1), (stage + kTileStages - 1) & (kTileStages - 1));
    const int so = stage * 2 * kTileOperand;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = fa[i][so + ((2 * q + g) ^ ka[i])];
        b[i] = fb[i][so + ((2 * q + g) ^ kb[i])];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32(a[i], b[j], acc[i][j]);
    }
  }
  wait_vmcnt<0>();  // nothing may still be on its way into LDS when the workgroup ends
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        store_logit(p, part, t0 + 64 * wm + 32 * i + acc_row(v, lane), e0 + 64 * wn + 32 * j + r, acc[i][j][v]);
}

// fp32 weights -> three bf16 planes [3][n] that add up to them, the smallest first.
__global__ __launch_bounds__(256) void gate_planes_kernel(const float* __restrict__ w, int64_t n8,
                                                          uint4* __restrict__ planes) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const float4* s = reinterpret_cast<const float4*>(w) + 2 * i;
  const Split3 v = split3(s[0], s[1]);
#pragma unroll
  for (int q = 0; q < 3; ++q) planes[(2 - q) * n8 + i] = v.f[q];
}

// logits = the partial sums in order, plus the bias.
__global__ __launch_bounds__(256) void gate_sum_kernel(const float* __restrict__ part, int parts, int64_t n, int E,
                                                       const float* __restrict__ bias, float* __restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  if (n % 4 == 0) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int q = 0; q < parts; ++q) {
      const float4 w = *reinterpret_cast<const float4*>(part + q * n + i);
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    if (bias) {
      v.x += bias[i % E];
      v.y += bias[(i + 1) % E];
      v.z += bias[(i + 2) % E];
      v.w += bias[(i + 3) % E];
    }
    *reinterpret_cast<float4*>(out + i) = v;
  } else {
    for (int64_t j = i; j < min(i + 4, n); ++j) {
      float v = 0.0f;
      for (int q = 0; q < parts; ++q) v += part[q * n + j];
      out[j] = bias ? v + bias[j % E] : v;
    }
  }
}

// Which kernel takes a call, and its workspace.
struct GatePlan {
  enum Kind { kDot, kSlice, kTile } kind;
  int slices, parts;
  size_t planes, total;  // bytes: offset of the weights' planes, and all of it
};

GatePlan gate_plan(int64_t T, int64_t H, int64_t E, bool w_bf16) {
  GatePlan g{GatePlan::kDot, 1, 1, 0, 0};
  if (T <= kDotTokens) return g;
  const int64_t big = (T + kTileRows - 1) / kTileRows * ((E + kTileRows - 1) / kTileRows);
  const int64_t small = (T + kSliceTile - 1) / kSliceTile * ((E + kSliceTile - 1) / kSliceTile);
  if (T <= 512 || H % 64 != 0) {
    g.kind = GatePlan::kSlice;
    // about a workgroup per CU, a multiple of the 8 XCDs, four K steps of 16 or more per wave
    const int64_t want = std::min<int64_t>((256 + small - 1) / small, H / 16 / (4 * kSliceWaves));
    g.slices = want >= 8 ? (int)std::min<int64_t>(want / 8 * 8, 32) : small < 256 ? (int)std::max<int64_t>(want, 1) : 1;
    g.parts = g.slices;
  } else {
    g.kind = GatePlan::kTile;
    const int planes = w_bf16 ? 1 : 3;
    const int64_t want = std::min<int64_t>(256 / (big * planes), H / 64 / 4);
    g.slices = (int)std::max<int64_t>(want, 1);
    g.parts = g.slices * planes;
  }
  if (g.parts > 1) g.total = ((size_t)g.parts * T * E * sizeof(float) + 255) / 256 * 256;
  g.planes = g.total;
  if (g.kind == GatePlan::kTile && !w_bf16) g.total += ((size_t)3 * E * H * 2 + 255) / 256 * 256;
  return g;
}

}  // namespace

size_t router_logits_workspace_bytes(int64_t T, int64_t H, int64_t E, bool w_bf16) {
  return gate_plan(T, H, E, w_bf16).total;
}

hipError_t launch_router_logits(const uint16_t* x, int64_t T, int H, const void* w, bool w_bf16, int E,
                                const float* bias, float* out, void* ws, hipStream_t s) {
  const GatePlan g = gate_plan(T, H, E, w_bf16);
  GateParams p{x, w, bias, g.parts > 1 ? static_cast<float*>(ws) : out, T, H, E, g.parts, g.slices};
  if (g.kind == GatePlan::kDot) {
    const int nt = T == 1 ? 1 : T == 2 ? 2 : 4;
    auto go = [&](auto kernel) { kernel<<<E, kDotThreads, 0, s>>>(p); };
    if (w_bf16)
      nt == 1 ? go(gate_dot_kernel<false, 1>) : nt == 2 ? go(gate_dot_kernel<false, 2>) : go(gate_dot_kernel<false, 4>);
    else
      nt == 1 ? go(gate_dot_kernel<true, 1>) : nt == 2 ? go(gate_dot_kernel<true, 2>) : go(gate_dot_kernel<true, 4>);
    return hipGetLastError();
  }
  if (g.kind == GatePlan::kSlice) {
    const int64_t tiles = (T + kSliceTile - 1) / kSliceTile * ((E + kSliceTile - 1) / kSliceTile);
    const dim3 grid((unsigned)(tiles * g.slices)), block(64 * kSliceWaves);
    w_bf16 ? gate_slice_kernel<false><<<grid, block, 0, s>>>(p) : gate_slice_kernel<true><<<grid, block, 0, s>>>(p);
  } else {
    if (!w_bf16) {
      uint4* planes = reinterpret_cast<uint4*>(static_cast<char*>(ws) + g.planes);
      const int64_t n8 = (int64_t)E * H / 8;
      gate_planes_kernel<<<(unsigned)((n8 + 255) / 256), 256, 0, s>>>(static_cast<const float*>(w), n8, planes);
      p.w = planes;
    }
    const int64_t items = (T + kTileRows - 1) / kTileRows * ((E + kTileRows - 1) / kTileRows) * g.parts;
    gate_tile_kernel<<<(unsigned)((items + 7) / 8 * 8), 256, 0, s>>>(p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.parts == 1) return e;
  const int64_t n = T * E;
  gate_sum_kernel<<<(unsigned)((n + 1023) / 1024), 256, 0, s>>>(static_cast<const float*>(ws), g.parts, n, E, bias,
                                                                out);
  return hipGetLastError();
}

}  // namespace nvfp4
