// Low-rank adapters of many requests beside a shared projection, on gfx950:
//   out[t][n] = y[t][n] + s[id] sum_j u[t][j] b[id][n][j],  u[t][j] = sum_k x[t][k] a[id][j][k]
// with id = ids[t], for tokens with an adapter (0 <= id < L); out = y for the
// others.  x, a, b are bf16; y and out bf16 or fp32.
//
// The tokens are grouped by adapter into tiles of up to 16 (one MFMA side), so
// an adapter is read once per 16 of its tokens instead of once per token.
// Two kernels: down (u, K long, r wide) and up (r long, N wide).  u is
// accumulated and kept in fp32; the up product takes it as a sum of bf16
// terms, each the rounding of what the ones before left: two for a bf16
// output (what is left is under 2^-16 of u, where the output's own rounding is
// 2^-8 of the sum), three for an fp32 output (2^-24).
#include <hip/hip_runtime.h>

#include "launch.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;  // tokens per tile

struct LoraParams {
  const void* y;       // [T][N], bf16 or fp32
  void* out;           // [T][N], the same type; may be y
  const uint16_t* x;   // [T][K]
  const uint16_t* a;   // [L][r][K]
  const uint16_t* b;   // [L][N][r]
  const int32_t* ids;  // [T]
  const float* scales; // nullable [L]
  int64_t T, N;
  int K, r, L;
  // grouping
  const GemmTile* tiles;
  const int* ntiles;
  const int* perm;     // sorted position -> token
  float* u;            // [sorted position][r], scaled
};

__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

// u of one tile: the waves take a slice of K each and their partial sums are
// added in order.  RT: 16-wide column tiles of r.
template <int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void lora_down_kernel(LoraParams p) {
  constexpr int kSteps = RT <= 2 ? 4 : 2;  // K steps of loads in flight
  constexpr int kCols = 16 * RT;
  __shared__ float part[WAVES][kTile * kCols];
  if ((int)blockIdx.x >= *p.ntiles) return;
  const GemmTile tile = p.tiles[blockIdx.x];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int64_t t = p.perm[tile.row0 + min(m, tile.nrows - 1)];
  const uint16_t* xr = p.x + t * p.K + 8 * g;
  const uint16_t* ar[RT];
#pragma unroll
  for (int c = 0; c < RT; ++c)
    ar[c] = p.a + ((int64_t)tile.expert * p.r + min(16 * c + m, p.r - 1)) * p.K + 8 * g;
  const int nk = p.K / 32, k0 = nk * wave / WAVES, k1 = nk * (wave + 1) / WAVES;
  f32x4 acc[RT];
#pragma unroll
  for (int c = 0; c < RT; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = k0; k < k1; k += kSteps) {
    uint4 xa[kSteps], wa[kSteps][RT];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int kk = 32 * min(k + i, k1 - 1);
      xa[i] = *reinterpret_cast<const uint4*>(xr + kk);
#pragma unroll
      for (int c = 0; c < RT; ++c) wa[i][c] = *reinterpret_cast<const uint4*>(ar[c] + kk);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (k + i < k1) {
#pragma unroll
        for (int c = 0; c < RT; ++c) acc[c] = mfma16(xa[i], wa[i][c], acc[c]);
      }
    }
  }
  // accumulator element i: token 4 g + i, column 16 c + lane % 16
#pragma unroll
  for (int c = 0; c < RT; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][(4 * g + i) * kCols + 16 * c + m] = acc[c][i];
  }
  __syncthreads();
  const float s = p.scales ? p.scales[tile.expert] : 1.0f;
  for (int i = threadIdx.x; i < kTile * kCols; i += 64 * WAVES) {
    const int row = i / kCols, col = i % kCols;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += part[w][i];
    if (row < tile.nrows && col < p.r) p.u[(int64_t)(tile.row0 + row) * p.r + col] = v * s;
  }
}

// Eight fp32 values -> TERMS bf16 fragments that add up to them.
template <int TERMS>
struct Terms {
  uint4 f[TERMS];
};
template <int TERMS>
__device__ __forceinline__ Terms<TERMS> split(const float4& a, const float4& b) {
  float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  Terms<TERMS> t;
#pragma unroll
  for (int q = 0; q < TERMS; ++q) {
    bf16x8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = (__bf16)v[i];
      v[i] -= (float)h[i];
    }
    t.f[q] = __builtin_bit_cast(uint4, h);
  }
  return t;
}

// out of one tile and 64 columns per wave.  The MFMA's rows are columns n of
// the output, its columns tokens: lane (token l % 16, g = l / 16) ends with
// the 16 consecutive n of its token from n0 + 16 g, so y and out move in
// 16-byte accesses and 128 bytes (bf16) of a row per wave.
constexpr int kUpWaves = 4;
constexpr int kUpCols = 64 * kUpWaves;

template <bool BF16>
__global__ __launch_bounds__(64 * kUpWaves) void lora_up_kernel(LoraParams p) {
  constexpr int TERMS = BF16 ? 2 : 3;
  const int ti = blockIdx.x;
  if (ti >= *p.ntiles) return;
  const GemmTile tile = p.tiles[ti];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * kUpCols + 64 * wave;
  if (n0 >= p.N) return;
  const bool valid = m < tile.nrows;
  const int row = tile.row0 + min(m, tile.nrows - 1);
  const int64_t t = p.perm[row];
  const int64_t nl = n0 + 16 * g;  // this lane's columns
  f32x4 acc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint16_t* br[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t n = min(n0 + 16 * (m >> 2) + 4 * q + (m & 3), p.N - 1);
    br[q] = p.b + ((int64_t)tile.expert * p.N + n) * p.r + 8 * g;
  }
  const float* ur = p.u + (int64_t)row * p.r + 8 * g;
  for (int j = 0; j < p.r; j += 32) {
    uint4 bq[4] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    float4 u0 = make_float4(0, 0, 0, 0), u1 = u0;
    if (j + 8 * g < p.r) {
#pragma unroll
      for (int q = 0; q < 4; ++q) bq[q] = *reinterpret_cast<const uint4*>(br[q] + j);
      u0 = *reinterpret_cast<const float4*>(ur + j);
      u1 = *reinterpret_cast<const float4*>(ur + j + 4);
    }
    const Terms<TERMS> us = split<TERMS>(u0, u1);
#pragma unroll
    for (int h = TERMS - 1; h >= 0; --h) {
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = mfma16(bq[q], us.f[h], acc[q]);
    }
  }
  if (!valid) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // eight columns at a time
    if (nl + 8 * h + 8 > p.N) continue;
    const int64_t o = t * p.N + nl + 8 * h;
    if constexpr (BF16) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.y) + o);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      bf16x8 r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[2 * i] = (__bf16)(bf16_lo(w[i]) + acc[2 * h + i / 2][2 * (i & 1)]);
        r[2 * i + 1] = (__bf16)(bf16_hi(w[i]) + acc[2 * h + i / 2][2 * (i & 1) + 1]);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + o) = __builtin_bit_cast(uint4, r);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.y) + o + 4 * i);
        const f32x4 c = acc[2 * h + i];
        v.x += c[0];
        v.y += c[1];
        v.z += c[2];
        v.w += c[3];
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o + 4 * i) = v;
      }
    }
  }
}

// out = y for the tokens without an adapter (not needed in place): row_bytes
// is a multiple of 16.
__global__ __launch_bounds__(256) void lora_copy_kernel(LoraParams p, int64_t row_bytes) {
  const int64_t t = blockIdx.x;
  const int id = p.ids[t];
  if (id >= 0 && id < p.L) return;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p.y) + t * row_bytes);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(p.out) + t * row_bytes);
  for (int64_t i = threadIdx.x; i < row_bytes / 16; i += 256) dst[i] = src[i];
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Layout {
  size_t u, offsets, perm, tiles, ntiles, err, route, total;
  int max_tiles;
};

Layout layout(int64_t T, int r, int L) {
  Layout l;
  l.max_tiles = (int)((T + kTile - 1) / kTile + (T < L ? T : L));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = up256(off + bytes);
    return at;
  };
  l.u = take(sizeof(float) * (size_t)T * r);
  l.offsets = take(sizeof(int) * (size_t)(L + 1));
  l.perm = take(sizeof(int) * (size_t)T);
  l.tiles = take(sizeof(GemmTile) * (size_t)l.max_tiles);
  l.ntiles = take(sizeof(int));
  l.err = take(sizeof(int));
  l.route = take(route_workspace_bytes(T, L));
  l.total = off;
  return l;
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int r, int L) { return layout(T, r, L).total; }

hipError_t launch_lora_add(const void* y, bool bf16, int64_t T, int64_t N, const uint16_t* x, int K,
                           const uint16_t* a, const uint16_t* b, int r, int L, const int32_t* ids,
                           const float* scales, void* out, void* ws, hipStream_t s) {
  const Layout l = layout(T, r, L);
  char* w = static_cast<char*>(ws);
  LoraParams p;
  p.y = y;
  p.out = out;
  p.x = x;
  p.a = a;
  p.b = b;
  p.ids = ids;
  p.scales = scales;
  p.T = T;
  p.N = N;
  p.K = K;
  p.r = r;
  p.L = L;
  GemmTile* tiles = reinterpret_cast<GemmTile*>(w + l.tiles);
  int* ntiles = reinterpret_cast<int*>(w + l.ntiles);
  int* perm = reinterpret_cast<int*>(w + l.perm);
  p.tiles = tiles;
  p.ntiles = ntiles;
  p.perm = perm;
  p.u = reinterpret_cast<float*>(w + l.u);
  hipError_t e = launch_route(ids, T, L, kTile, 0, kTile, reinterpret_cast<int*>(w + l.offsets), perm, tiles, ntiles,
                              nullptr, nullptr, reinterpret_cast<int*>(w + l.err),
                              reinterpret_cast<int*>(w + l.route), nullptr, s);
  if (e != hipSuccess) return e;
  const int rt = (r + 15) / 16;
  if (rt == 1)
    lora_down_kernel<1, 16><<<l.max_tiles, 64 * 16, 0, s>>>(p);
  else if (rt == 2)
    lora_down_kernel<2, 16><<<l.max_tiles, 64 * 16, 0, s>>>(p);
  else if (rt <= 4)
    lora_down_kernel<4, 8><<<l.max_tiles, 64 * 8, 0, s>>>(p);
  else
    lora_down_kernel<8, 8><<<l.max_tiles, 64 * 8, 0, s>>>(p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const dim3 blocks((unsigned)l.max_tiles, (unsigned)((N + kUpCols - 1) / kUpCols));
  if (bf16)
    lora_up_kernel<true><<<blocks, 64 * kUpWaves, 0, s>>>(p);
  else
    lora_up_kernel<false><<<blocks, 64 * kUpWaves, 0, s>>>(p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (out != y) lora_copy_kernel<<<(unsigned)T, 256, 0, s>>>(p, N * (bf16 ? 2 : 4));
  return hipGetLastError();
}

}  // namespace nvfp4
