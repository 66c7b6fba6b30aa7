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
#include <cmath>

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

__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
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

// ---- up to eight tokens: a workgroup per expert, every thread a few 16-byte
// chunks of the row, all of them requested at once: one launch that lasts one
// trip to memory (T1 H7168 E256: 3.0 us for 3.7 MB, T8 5.9).  fp32 fused
// multiply-adds keep the products exact.
constexpr int kDotThreads = 256;
constexpr int kDotTokens = 8;

template <bool F32W, int NT>
__global__ __launch_bounds__(kDotThreads) void gate_dot_kernel(GateParams p) {
  constexpr int kUnroll = NT <= 2 ? 4 : 1;
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
// registers.  2 x 2 MFMA tiles of 16 x 16, whose loads take 64 bytes of 16 rows
// each.  Workgroups that run on one XCD (blockIdx % 8) take the same slices, so
// an XCD's L2 fetches its part of x and w and not all of both.  The loop is
// short: such a call spends most of its time on trips to memory, and fetching
// its code is one of them.  Batches of 8, 4, 2 and 1 steps of loads take 8.3,
// 6.5, 5.7 and 5.6 us for T256 H2048 E64, 8.7, 8.7, 8.1 and 8.0 for T128 H7168
// E256 with operands in the caches; two keep more in flight from memory.
constexpr int kSliceWaves = 4;
constexpr int kSliceTile = 32;

template <bool F32W>
__global__ __launch_bounds__(64 * kSliceWaves) void gate_slice_kernel(GateParams p) {
  constexpr int kSteps = 2;  // K steps of 32 per batch of loads
  __shared__ float part[kSliceWaves][32 * 33];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int etiles = (p.E + kSliceTile - 1) / kSliceTile;
  const int slice = blockIdx.x % p.slices, tile = blockIdx.x / p.slices;
  const int e0 = tile % etiles * kSliceTile;
  const int64_t t0 = (int64_t)(tile / etiles) * kSliceTile;
  const int r = lane & 15, g = lane >> 4;
  const uint16_t* xr[2];
  int64_t wo[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    xr[h] = p.x + min(t0 + 16 * h + r, p.T - 1) * p.H + 8 * g;
    wo[h] = (int64_t)min(e0 + 16 * h + r, p.E - 1) * p.H + 8 * g;
  }
  const int nk = p.H / 32, share = p.slices * kSliceWaves, mine = slice * kSliceWaves + wave;
  const int k0 = (int)((uint32_t)(nk * mine) / (uint32_t)share), k1 = (int)((uint32_t)(nk * (mine + 1)) / (uint32_t)share);
  f32x4 acc[2][2] = {};  // [token half][expert half]
  for (int k = k0; k < k1; k += kSteps) {
    uint4 a[kSteps][2];
    if constexpr (F32W) {
      float4 b[kSteps][2][2];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int kk = 32 * min(k + i, k1 - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[i][h] = *reinterpret_cast<const uint4*>(xr[h] + kk);
          const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + wo[h] + kk);
          b[i][h][0] = s[0];
          b[i][h][1] = s[1];
        }
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (k + i < k1) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const Split3 s = split3(b[i][e][0], b[i][e][1]);
#pragma unroll
            for (int q = 2; q >= 0; --q)
#pragma unroll
              for (int t = 0; t < 2; ++t) acc[t][e] = mfma16(a[i][t], s.f[q], acc[t][e]);
          }
        }
      }
    } else {
      uint4 b[kSteps][2];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int kk = 32 * min(k + i, k1 - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[i][h] = *reinterpret_cast<const uint4*>(xr[h] + kk);
          b[i][h] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.w) + wo[h] + kk);
        }
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (k + i < k1) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) acc[t][e] = mfma16(a[i][t], b[i][e], acc[t][e]);
        }
      }
    }
  }
  // accumulator element i: token 4 g + i, expert lane % 16 of its tile
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][33 * (16 * t + 4 * g + i) + 16 * e + r] = acc[t][e][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * 32; i += 64 * kSliceWaves) {
    const int row = i >> 5, col = i & 31;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kSliceWaves; ++w) v += part[w][33 * row + col];
    store_logit(p, slice, t0 + row, e0 + col, v);
  }
}

// ---- many tokens: 128 tokens x 128 experts per workgroup, K in steps of 64
// through four LDS stages filled by direct loads.  Of the eight waves four
// take the first half of every step and four the second, 64 x 64 outputs each
// (2 x 2 MFMA tiles), and the halves are added at the end; the fragments of
// the next step are read before this step's MFMAs.  Chunk c (16 bytes) of a row
// lies at c ^ swz_key(row).  The experts are the MFMA's rows, so that a lane
// ends with four experts of one token in a register quad, which is one store.
// The direct loads alone (32 KiB a step and CU) take 48 of the 71 to 75 us of
// T16384 H7168 E256 on repeated inputs, part of which stay in the 256 MB cache,
// and 77 of the 80 us on changing ones.  64 x 128 outputs per wave over
// quarters of a step, a quarter less LDS traffic, gain 1 % there and lose 10 %
// below 4096 tokens.  The time outside the loop counts as well: an epilogue that
// sent all sums through LDS and stored single floats took 16000 cycles.
// With too few tiles for the chip, K is sliced as well; an fp32 weight comes as
// three bf16 planes (gate_planes_kernel), each a partial sum of its own.
constexpr int kTileRows = 128;
constexpr int kTileStages = 4;
constexpr int kTileOperand = kTileRows * 8;  // 16-byte chunks of one operand's stage

__global__ __launch_bounds__(512) void gate_tile_kernel(GateParams p) {
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
  const int s0 = (int)((uint32_t)(steps * slice) / (uint32_t)p.slices);
  const int s1 = (int)((uint32_t)(steps * (slice + 1)) / (uint32_t)p.slices);
  const uint32_t row_bytes = 2u * (uint32_t)p.H;
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(p.x) + t0 * row_bytes;
  const uint8_t* wb = static_cast<const uint8_t*>(p.w) + ((int64_t)plane * p.E + e0) * row_bytes;
  const int trows = (int)min((int64_t)kTileRows, p.T - t0), erows = min(kTileRows, p.E - e0);
  // load u of a wave: rows 16 wave + 8 u .. + 7 of each operand, 128 bytes each
  uint32_t xo[2], wo[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int row = 16 * wave + 8 * u + (lane >> 3);
    const uint32_t chunk = 16u * (uint32_t)((lane & 7) ^ swz_key(row));
    xo[u] = (uint32_t)min(row, trows - 1) * row_bytes + chunk;  // rows past the end repeat the last one
    wo[u] = (uint32_t)min(row, erows - 1) * row_bytes + chunk;
  }
  auto load = [&](int step, int stage) {
    uint4* dst = lds + stage * 2 * kTileOperand + 16 * 8 * wave;
    const size_t at = (size_t)step * 128;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      dma16s(reinterpret_cast<f16x8*>(dst + 64 * u), xb + at, xo[u]);
      dma16s(reinterpret_cast<f16x8*>(dst + kTileOperand + 64 * u), wb + at, wo[u]);
    }
  };
  // rows 32 i + r of either operand, chunks 4 half + 2 q + g; the key of a row
  // depends on r and on the parity of i, and chunk c ^ 2 lies at address ^ 2
  const int half = wave >> 2, wm = (wave >> 1) & 1, wn = wave & 1, r = lane & 31, g = lane >> 5;
  const int c0 = (4 * half + g) ^ swz_key(r), c1 = (4 * half + g) ^ swz_key(32 + r);
  const uint4* const fx = lds + 8 * (64 * wm + r);
  const uint4* const fw = lds + kTileOperand + 8 * (64 * wn + r);
  struct Frags {
    uint4 x[2][2], w[2][2];  // [q][i]
  };
  auto read = [&](int stage, Frags& f) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = stage * 2 * kTileOperand + 256 * i + ((i ? c1 : c0) ^ (2 * q));
        f.x[q][i] = fx[at];
        f.w[q][i] = fw[at];
      }
  };
  f32x16 acc[2][2] = {};  // [token tile][expert tile]
  // One step: its fragments are in cur.  The barrier publishes the stage of
  // the next step and ends every wave's reads of this one's, which the load of
  // step s + 4 then fills; 4 loads a step, so with at most 8 on their way all
  // but those of steps s + 2 and s + 3 have landed.
  auto body = [&](int s, const Frags& cur, Frags& nxt) {
    const int stage = (s - s0) & (kTileStages - 1);
    wait_vmcnt<8>();
    lds_barrier();
    SCHED_FENCE();
    read((stage + 1) & (kTileStages - 1), nxt);
    load(min(s + kTileStages, s1 - 1), stage);
    SCHED_FENCE();
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32(cur.w[q][j], cur.x[q][i], acc[i][j]);
    SCHED_FENCE();
  };
#pragma unroll
  for (int i = 0; i < kTileStages; ++i) load(min(s0 + i, s1 - 1), i);
  Frags even, odd;
  wait_vmcnt<12>();
  lds_barrier();
  read(0, even);
  for (int s = s0;;) {
    body(s, even, odd);
    if (++s == s1) break;
    body(s, odd, even);
    if (++s == s1) break;
  }
  wait_vmcnt<0>();  // the last loads go into stages that nobody reads any more
  // Each half hands one token tile's sums to the other and keeps the other
  // tile (first half: token tile 0): 8 KiB of LDS per wave, quad by quad
  f32x4* const sum = reinterpret_cast<f32x4*>(lds);
  auto quad = [](const f32x16& v, int i) { return f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]}; };
  __syncthreads();
  f32x16 keep[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    keep[j] = half ? acc[1][j] : acc[0][j];
    const f32x16 give = half ? acc[0][j] : acc[1][j];
#pragma unroll
    for (int v = 0; v < 4; ++v) sum[512 * wave + 64 * (4 * j + v) + lane] = quad(give, v);
  }
  __syncthreads();
  const int64_t t = t0 + 64 * wm + 32 * half + r;
  float* const out = p.out + ((int64_t)part * p.T + t) * p.E;
  const bool vec = p.E % 4 == 0, biased = p.parts == 1 && p.bias;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const f32x4 o = sum[512 * (wave ^ 4) + 64 * (4 * j + v) + lane];
      f32x4 y = quad(keep[j], v);
      y = half ? o + y : y + o;  // the first half of K first
      const int e = e0 + 64 * wn + 32 * j + 8 * v + 4 * g;
      if (t >= p.T || e >= p.E) continue;
      if (vec) {
        if (biased) y += f32x4{p.bias[e], p.bias[e + 1], p.bias[e + 2], p.bias[e + 3]};
        *reinterpret_cast<f32x4*>(out + e) = y;
      } else {
        for (int u = 0; u < 4; ++u)
          if (e + u < p.E) out[e + u] = biased ? y[u] + p.bias[e + u] : y[u];
      }
    }
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
      const uint32_t e = (uint32_t)i % (uint32_t)E;  // at most 2^29 logits
      float* y = &v.x;
#pragma unroll
      for (int u = 0; u < 4; ++u) y[u] += bias[e + u < (uint32_t)E ? e + u : (e + u) % (uint32_t)E];
    }
    *reinterpret_cast<float4*>(out + i) = v;
  } else {
    for (int64_t j = i; j < min(i + 4, n); ++j) {
      float v = 0.0f;
      for (int q = 0; q < parts; ++q) v += part[q * n + j];
      out[j] = bias ? v + bias[(uint32_t)j % (uint32_t)E] : v;
    }
  }
}

// Which kernel takes a call, and its workspace.  Measured (us of GPU time):
// dot against slices (H7168 E256) at 8 tokens 5.9 / 6.7, at 12 tokens 9.4 / 6.4
// (with 16 tokens per workgroup); slices against tiles by the slices' work,
// small tiles x H: bf16 H7168 E256 at 256 tokens (0.46 M) 11.7 / 14.0, at 300
// (0.57 M) 14.8 / 13.9; H4096 E72 at 1024 (0.39 M) 10.6 / 12.2, at 2048 (0.79 M)
// 16.8 / 13.2; fp32, whose tiles cost three times as much, H7168 E256 at 384 (0.69
// M) 20.1 / 23.1, at 512 (0.92 M) 24.7 / 22.6, H4096 E72 at 2048 21.6 / 20.8.
// The tiles' steps are 64 wide, so that an H of 32 beyond a multiple of 64 goes
// to the slices at any size, which costs with many tokens: H7136 against H7168
// (E256, bf16 / fp32) at 1024 tokens 27 / 39 against 20 / 30, at 4096 100 / 133
// against 30 / 77, at 16384 396 / 522 against 85 / 240 (a product of fp32 copies
// in the library: 517 / 506).  Padding H with zeros, once in w, avoids it.
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
  if (H % 64 != 0 || small * H <= (w_bf16 ? 1 << 19 : 11 << 16)) {
    g.kind = GatePlan::kSlice;
    // about a workgroup per CU and two K steps of 32 or more per wave;
    // multiples of the 8 XCDs, or with a short K a power of two
    const int64_t want = std::min<int64_t>((256 + small - 1) / small, H / 16 / (4 * kSliceWaves));
    if (want >= 8)
      g.slices = (int)std::min<int64_t>(want / 8 * 8, 32);
    else if (small <= 256)
      g.slices = H >= 4096 ? 8 : want >= 4 ? 4 : want >= 2 ? 2 : 1;
    g.parts = g.slices;
  } else {
    g.kind = GatePlan::kTile;
    const int planes = w_bf16 ? 1 : 3;
    // as many slices as fill the chip, unless the partial sums cost more than
    // the shorter loops save: a step takes 0.45 us, a partial logit 8 bytes
    // written and read at 5 TB/s, so that steps / n * 0.45 us + n * T E * 1.6 ps
    // is least at n^2 = 4400 H / (T E)
    const int64_t want = std::min<int64_t>({256 / (big * planes), H / 64 / 4,
                                            (int64_t)std::sqrt(4400.0 * H / ((double)T * E * planes))});
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
    auto go = [&](auto one, auto two, auto four, auto eight) {
      (T == 1 ? one : T == 2 ? two : T <= 4 ? four : eight)<<<E, kDotThreads, 0, s>>>(p);
    };
    if (w_bf16)
      go(gate_dot_kernel<false, 1>, gate_dot_kernel<false, 2>, gate_dot_kernel<false, 4>, gate_dot_kernel<false, 8>);
    else
      go(gate_dot_kernel<true, 1>, gate_dot_kernel<true, 2>, gate_dot_kernel<true, 4>, gate_dot_kernel<true, 8>);
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
    gate_tile_kernel<<<(unsigned)((items + 7) / 8 * 8), 512, 0, s>>>(p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.parts == 1) return e;
  const int64_t n = T * E;
  gate_sum_kernel<<<(unsigned)((n + 1023) / 1024), 256, 0, s>>>(static_cast<const float*>(ws), g.parts, n, E, bias,
                                                                out);
  return hipGetLastError();
}

}  // namespace nvfp4
