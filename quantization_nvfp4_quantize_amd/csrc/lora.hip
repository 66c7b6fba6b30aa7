// Low-rank adapters of many requests beside a shared projection, on gfx950:
//   out[t][n] = y[t][n] + s[id] sum_j u[t][j] b[id][n][j],  u[t][j] = sum_k x[t][k] a[id][j][k]
// with id = ids[t], for tokens with an adapter (0 <= id < L); out = y for the
// others.  x, a, b are bf16; y and out bf16 or fp32.
//
// The tokens are grouped by adapter into tiles, so that an adapter is read once
// per tile and not once per token.  Two kernels: down (u: K long, r wide) and
// up (r long, N wide).  u is accumulated and kept in fp32, as partial sums over
// slices of K where the tiles alone do not fill the chip; the up kernel adds the
// slices and takes u as a sum of bf16 terms, each the rounding of what the
// ones before left: two for a bf16 output (what is left is under 2^-16 of u,
// where the output's own rounding is 2^-8 of the sum), three for an fp32
// output (2^-24).  A token's result does not depend on its place in a tile.
//
// Up to kLeaderTokens tokens the down kernel finds the groups by itself; up to
// kGroupTokens one workgroup groups them; beyond, the grouping of the expert
// FFN does.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gemm_common.hpp"
#include "launch.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kLeaderTokens = 256;
constexpr int kGroupTokens = 16384;
// Tokens per tile: kTileRows where the adapters have many tokens each,
// kFewRows (one MFMA side) else
constexpr int kTileRows = 64, kFewRows = 16;

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
  int slices;          // slices of K
  int tile_rows;       // tokens per tile
  // grouping: tiles of one adapter (expert), or of tokens without one (-1)
  GemmTile* tiles;
  int* ntiles;
  int* perm;           // tile position -> token
  float* u;            // [slice][token][r], scaled
};

__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

__device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

// The tokens of the tile that token t leads: t has an adapter, and a multiple
// of kFewRows tokens before t share it; the tile is t and the next ones of
// that adapter.  Every workgroup of t comes to the same answer from the ids
// alone.  Returns the number of tokens (0: t leads nothing), their indices in
// tok.  kLeaderTokens threads or more.
__device__ __forceinline__ int lead(const LoraParams& p, int t, int* tok, uint64_t* masks) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int id = p.ids[t];
  const bool same = tid < p.T && p.ids[tid] == id;
  const uint64_t mine = __ballot(same);
  if (lane == 0 && wave < kLeaderTokens / 64) masks[wave] = mine;
  __syncthreads();
  if (id < 0 || id >= p.L) return 0;
  const uint64_t below = lane ? ~0ull >> (64 - lane) : 0ull;
  int before = 0, to_t = 0, all = 0;  // matches before this thread's token, before t, and in all
#pragma unroll
  for (int w = 0; w < kLeaderTokens / 64; ++w) {
    const uint64_t m = masks[w];
    const int n = __popcll(m);
    all += n;
    if (w < wave) before += n;
    if (w < (t >> 6)) to_t += n;
    if (w == (t >> 6)) to_t += __popcll(m & ((t & 63) ? ~0ull >> (64 - (t & 63)) : 0ull));
  }
  if (to_t % kFewRows) return 0;
  before += __popcll(mine & below);
  if (same && before >= to_t && before < to_t + kFewRows) tok[before - to_t] = tid;
  __syncthreads();
  return min(all - to_t, kFewRows);
}

// u of 16 tokens and one slice of K, a share of the slice per wave, operands
// straight from memory.  RT: 16-wide column tiles of r.  LEADER: the tile is
// the one token blockIdx.y leads, and slice 0 lists it for the up kernel; else
// rows 16 blockIdx.z .. of tile blockIdx.y.
// 128 tokens of 64 adapters, K 4096, r 16: 5.7 us for 9 MB, one trip to memory
// for the ids and one or two for the operands.
constexpr int kDirectWaves = 4;

template <int RT, bool LEADER>
__global__ __launch_bounds__(64 * kDirectWaves) void lora_down_direct_kernel(LoraParams p) {
  constexpr int WAVES = kDirectWaves;
  constexpr int kSteps = 2;  // K steps of 32 per batch of loads (8 and 4: up to 4 % slower, by their code)
  constexpr int kCols = 16 * RT;
  __shared__ float part[WAVES][16 * kCols];
  __shared__ int tok[16];
  __shared__ uint64_t masks[kLeaderTokens / 64];
  const int slice = blockIdx.x, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int id, rows;
  if constexpr (LEADER) {
    const int t = blockIdx.y;
    rows = lead(p, t, tok, masks);
    id = p.ids[t];
    if (slice == 0) {
      const bool bare = id < 0 || id >= p.L;
      if (threadIdx.x == 0) p.tiles[t] = GemmTile{bare ? -1 : id, kFewRows * t, bare ? 1 : rows, 0};
      if (threadIdx.x < (unsigned)max(rows, 1)) p.perm[kFewRows * t + threadIdx.x] = rows ? tok[threadIdx.x] : t;
    }
    if (rows == 0) return;
  } else {
    if ((int)blockIdx.y >= *p.ntiles) return;
    const GemmTile tile = p.tiles[blockIdx.y];
    id = tile.expert;
    rows = min(tile.nrows - 16 * (int)blockIdx.z, 16);
    if (id < 0 || rows <= 0) return;
    if (threadIdx.x < 16)
      tok[threadIdx.x] = p.perm[tile.row0 + 16 * blockIdx.z + min((int)threadIdx.x, rows - 1)];
    __syncthreads();
  }
  const int m = lane & 15, g = lane >> 4;
  const uint16_t* xr = p.x + (int64_t)tok[min(m, rows - 1)] * p.K + 8 * g;
  const uint16_t* ar[RT];
#pragma unroll
  for (int c = 0; c < RT; ++c) ar[c] = p.a + ((int64_t)id * p.r + min(16 * c + m, p.r - 1)) * p.K + 8 * g;
  const int nk = p.K / 32, share = WAVES * p.slices, mine = WAVES * slice + wave;
  const int k0 = (int)((uint32_t)(nk * mine) / (uint32_t)share);
  const int k1 = (int)((uint32_t)(nk * (mine + 1)) / (uint32_t)share);
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
  const float s = p.scales ? p.scales[id] : 1.0f;
  for (int i = threadIdx.x; i < 16 * kCols; i += 64 * WAVES) {
    const int row = i / kCols, col = i % kCols;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += part[w][i];
    if (row < rows && col < p.r) p.u[((int64_t)slice * p.T + tok[row]) * p.r + col] = v * s;
  }
}

// u of one tile of 64 tokens and one slice of K in steps of 64 through four LDS
// stages filled by direct loads.  Wave w: tokens 32 (w & 1) .. + 31, the K half
// w / 2 of every step, all of r (R32 MFMA tiles of 32); the halves are added
// at the end.  Chunk c (16 bytes) of a row lies at c ^ swz_key(row).  The rows
// of a are the MFMA's rows: a lane ends with four columns of u of one token.
// Bound by x: 5003 tokens, K 7168, r 64 in 19 us (72 MB), 4096 tokens, K 4096, r 32
// in 8.5 us (28 MB).
constexpr int kDownStages = 4;

template <int R32>
__global__ __launch_bounds__(256) void lora_down_tile_kernel(LoraParams p) {
  constexpr int kX = kTileRows * 8, kStage = kX + 32 * R32 * 8;  // 16-byte chunks
  __shared__ uint4 lds[kDownStages * kStage];
  if ((int)blockIdx.y >= *p.ntiles) return;
  const GemmTile tile = p.tiles[blockIdx.y];
  if (tile.expert < 0) return;
  const int slice = blockIdx.x, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = p.K / 64;
  const int s0 = (int)((uint32_t)(steps * slice) / (uint32_t)p.slices);
  const int s1 = (int)((uint32_t)(steps * (slice + 1)) / (uint32_t)p.slices);
  // load u of a wave: x rows 16 wave + 8 u .. + 7 (through perm), a rows 8 R32 wave + 8 u .. + 7
  const uint8_t* xs[2];
  const uint8_t* as[R32];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int row = 16 * wave + 8 * u + (lane >> 3);
    const int64_t t = p.perm[tile.row0 + min(row, tile.nrows - 1)];  // rows past the end repeat the last one
    xs[u] = reinterpret_cast<const uint8_t*>(p.x + t * p.K) + 16 * ((lane & 7) ^ swz_key(row));
  }
#pragma unroll
  for (int u = 0; u < R32; ++u) {
    const int row = 8 * R32 * wave + 8 * u + (lane >> 3);
    as[u] = reinterpret_cast<const uint8_t*>(p.a + ((int64_t)tile.expert * p.r + min(row, p.r - 1)) * p.K) +
            16 * ((lane & 7) ^ swz_key(row));
  }
  auto load = [&](int step, int stage) {
    uint4* dst = lds + stage * kStage;
    const size_t at = (size_t)step * 128;
#pragma unroll
    for (int u = 0; u < 2; ++u) dma16(reinterpret_cast<f16x8*>(dst + 8 * (16 * wave + 8 * u)), xs[u] + at);
#pragma unroll
    for (int u = 0; u < R32; ++u)
      dma16(reinterpret_cast<f16x8*>(dst + kX + 8 * (8 * R32 * wave + 8 * u)), as[u] + at);
  };
  const int half = wave >> 1, tm = wave & 1, r = lane & 31, g = lane >> 5;
  // the key of row 32 i + r depends on r and on the parity of i; chunk c ^ 2
  // lies at address ^ 2
  const int key0 = (4 * half + g) ^ swz_key(r), key1 = (4 * half + g) ^ swz_key(32 + r);
  f32x16 acc[R32] = {};
#pragma unroll
  for (int i = 0; i < kDownStages - 1; ++i) load(min(s0 + i, s1 - 1), i);
  for (int s = s0; s < s1; ++s) {
    const int stage = (s - s0) & (kDownStages - 1);
    // 2 + R32 loads a step; two later steps may still be on their way
    wait_vmcnt<2 * (2 + R32)>();
    lds_barrier();  // stage s has landed for every wave, and every wave has read stage s - 1
    load(min(s + kDownStages - 1, s1 - 1), (stage + kDownStages - 1) & (kDownStages - 1));
    const uint4* fx = lds + stage * kStage + 8 * (32 * tm + r);
    const uint4* fa = lds + stage * kStage + kX + 8 * r;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 xf = fx[(tm ? key1 : key0) ^ (2 * q)];
#pragma unroll
      for (int c = 0; c < R32; ++c) acc[c] = mfma32(fa[256 * c + (((c & 1) ? key1 : key0) ^ (2 * q))], xf, acc[c]);
    }
  }
  wait_vmcnt<0>();  // the last loads go into stages that nobody reads any more
  __syncthreads();
  f32x4* const sum = reinterpret_cast<f32x4*>(lds) + 256 * R32 * tm + lane;
  if (half) {
#pragma unroll
    for (int c = 0; c < R32; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        sum[64 * (4 * c + v)] = f32x4{acc[c][4 * v], acc[c][4 * v + 1], acc[c][4 * v + 2], acc[c][4 * v + 3]};
  }
  __syncthreads();
  const int row = 32 * tm + r;
  if (half || row >= tile.nrows) return;
  const float f = p.scales ? p.scales[tile.expert] : 1.0f;
  float* const u = p.u + ((int64_t)slice * p.T + p.perm[tile.row0 + row]) * p.r;
#pragma unroll
  for (int c = 0; c < R32; ++c)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int j = 32 * c + 8 * v + 4 * g;
      const f32x4 y =
          (f32x4{acc[c][4 * v], acc[c][4 * v + 1], acc[c][4 * v + 2], acc[c][4 * v + 3]} + sum[64 * (4 * c + v)]) * f;
      if (j < p.r) *reinterpret_cast<f32x4*>(u + j) = y;
    }
}

// Groups up to kGroupTokens tokens by adapter, one workgroup of 1024 threads:
// a histogram in LDS, a scan, and each token's place from a second count.  The
// places inside an adapter depend on the order of the atomics, which changes
// no result.  Tokens without an adapter come last, in tiles of expert -1.  The
// ids are requested four at a time and kept in LDS for the second count: the
// kernel lasts as long as its chain of loads (6 us for 4096 tokens).
__global__ __launch_bounds__(1024) void lora_group_kernel(LoraParams p) {
  __shared__ int count[513], place[513], wsum[16];
  __shared__ uint16_t adapter[kGroupTokens];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, T = (int)p.T;
  if (tid <= p.L) count[tid] = 0;
  __syncthreads();
  // one count per wave where its 64 tokens share an adapter
  auto add = [&](int* c, int id) {
    const int first = __builtin_amdgcn_readfirstlane(id);
    if (__ballot(id != first) == 0) {
      const uint64_t all = __ballot(true);
      int base = 0;
      if (lane == 0) base = atomicAdd(&c[first], __popcll(all));
      return __builtin_amdgcn_readfirstlane(base) + lane;
    }
    return atomicAdd(&c[id], 1);
  };
  for (int t0 = tid; t0 < T; t0 += 4 * 1024) {
    int id[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) id[i] = p.ids[min(t0 + 1024 * i, T - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 1024 * i;
      if (t >= T) break;
      const int e = id[i] < 0 || id[i] >= p.L ? p.L : id[i];
      adapter[t] = (uint16_t)e;
      add(count, e);
    }
  }
  __syncthreads();
  // tokens (low half) and tiles (high half) of the adapters before this one
  const int n = tid <= p.L ? count[tid] : 0, tiles = (n + p.tile_rows - 1) / p.tile_rows;
  const int v = n | tiles << 16;
  int x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  if (lane == 63) wsum[wave] = x;
  __syncthreads();
  for (int w = 0; w < wave; ++w) x += wsum[w];
  if (tid <= p.L) {
    const int start = (x - v) & 0xffff, first = (x - v) >> 16;
    place[tid] = start;
    for (int i = 0; i < tiles; ++i)
      p.tiles[first + i] =
          GemmTile{tid == p.L ? -1 : tid, start + i * p.tile_rows, min(p.tile_rows, n - i * p.tile_rows), 0};
    if (tid == p.L) *p.ntiles = first + tiles;
  }
  __syncthreads();
  for (int t = tid; t < T; t += 1024) p.perm[add(place, adapter[t])] = t;
}

// Eight fp32 values -> TERMS bf16 fragments that add up to them; an infinite
// value is its first term.  A finite value beyond the largest bf16 (it would
// round to infinity) leaves the excess to the next term.
template <int TERMS>
struct Terms {
  uint4 f[TERMS];
};
template <int TERMS>
__device__ __forceinline__ Terms<TERMS> split(const f32x4& a, const f32x4& b) {
  constexpr float kMost = 0x1.fep127f;
  float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  Terms<TERMS> t;
#pragma unroll
  for (int q = 0; q < TERMS; ++q) {
    bf16x8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (q == 0) {  // what it leaves is finite and small
        const bool finite = __builtin_fabsf(v[i]) < INFINITY;
        h[i] = (__bf16)(finite ? __builtin_amdgcn_fmed3f(v[i], -kMost, kMost) : v[i]);
        v[i] = finite ? v[i] - (float)h[i] : 0.0f;  // not inf - inf
      } else {
        h[i] = (__bf16)v[i];
        v[i] -= (float)h[i];
      }
    }
    t.f[q] = __builtin_bit_cast(uint4, h);
  }
  return t;
}

// out of one tile.  The workgroup adds the slices of u once and keeps its terms
// in LDS as MFMA fragments; then each wave walks over 64-column chunks of the
// output.  The MFMA's rows are columns of the output, its columns tokens: lane
// (token l % 16, g = l / 16) ends with columns col_of(q, 4 g + i) of its token in
// element i of accumulator q, 16 bytes at a time, and the four g of a token with
// 64 adjacent bytes per access; an adapter's rows of b are loaded once for the
// tile.  Bound by y and out: 61 us of the 78 for 4096 tokens, N 16384, r 32, bf16
// are this kernel's, 268 MB at 4.4 TB/s.  Tiles of tokens without an adapter go
// the same way without a product (a loop token by token over them, 11 tiles of
// the 75, took 70 us longer than all the others).  Workgroups of one tile are
// launched next to each other: launched tile by tile within a chunk the same
// call takes 5 us more, in runs of tiles per XCD 6 us more.
constexpr int kUpWaves = 4;

// Column (of 64) of row m of MFMA tile q: for a bf16 output tiles 2 h and 2 h + 1
// make eight adjacent columns of a lane, for fp32 each tile makes four.
template <bool BF16>
__device__ __forceinline__ int col_of(int q, int m) {
  return BF16 ? 32 * (q >> 1) + 8 * (m >> 2) + 4 * (q & 1) + (m & 3) : 16 * q + m;
}

// Eight bf16 values plus eight fp32 ones, rounded once.
__device__ __forceinline__ uint4 add_bf16(const uint4& v, const f32x4& lo, const f32x4& hi) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float d[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = (__bf16)(bf16_lo(w[i]) + d[2 * i]);
    r[2 * i + 1] = (__bf16)(bf16_hi(w[i]) + d[2 * i + 1]);
  }
  return __builtin_bit_cast(uint4, r);
}

// RC: 32-wide chunks of r; MT: MFMA tiles of 16 tokens per tile.  Columns and
// offsets inside an adapter fit 32 bits (N <= 2^20, r <= 128).
template <bool BF16, int RC, int MT>
__device__ __forceinline__ void lora_up(const LoraParams& p) {
  constexpr int TERMS = BF16 ? 2 : 3;
  constexpr int kSize = BF16 ? 2 : 4;
  constexpr int PIECES = BF16 ? 2 : 4;  // 16-byte accesses of a lane per token and chunk, 64 bytes apart
  __shared__ uint4 us[MT * RC * TERMS][64];
  if (p.ntiles && (int)blockIdx.y >= *p.ntiles) return;
  const GemmTile tile = p.tiles[blockIdx.y];
  if (tile.nrows == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int N = (int)p.N, r = p.r;
  const int n_first = ((int)blockIdx.x * kUpWaves + wave) * 64, n_step = (int)gridDim.x * kUpWaves * 64;
  const bool bare = tile.expert < 0;  // tokens without an adapter: out = y
  if (bare && p.out == p.y) return;
  int64_t row[MT];  // byte offset of this lane's token
#pragma unroll
  for (int i = 0; i < MT; ++i)
    row[i] = p.perm[tile.row0 + min(16 * i + m, tile.nrows - 1)] * (p.N * kSize) + 16 * g;
  const char* const yb = static_cast<const char*>(p.y);
  char* const ob = static_cast<char*>(p.out);
  // 16 bytes of y from byte 64 h of the chunk at column n on; past the end of
  // the row (whole pieces, N % 8 == 0) the last ones again
  auto load_y = [&](int i, int h, int n) {
    const int at = min(n * kSize + 64 * h, N * kSize - 16 - 16 * g);
    return *reinterpret_cast<const uint4*>(yb + row[i] + at);
  };
  auto inside = [&](int h, int n) { return n * kSize + 64 * h + 16 * g < N * kSize; };
  if (bare) {
    for (int n = n_first; n < N; n += n_step) {
      uint4 y[MT][PIECES];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < PIECES; ++h) y[i][h] = load_y(i, h, n);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < PIECES; ++h)
          if (16 * i + m < tile.nrows && inside(h, n))
            *reinterpret_cast<uint4*>(ob + row[i] + n * kSize + 64 * h) = y[i][h];
    }
    return;
  }
  for (int w = wave; w < MT * RC; w += kUpWaves) {
    const int i = w / RC, c = w % RC;
    if (16 * i >= tile.nrows) break;
    f32x4 u0 = {0.0f, 0.0f, 0.0f, 0.0f}, u1 = u0;
    if (32 * c + 8 * g < r) {
      const float* ur = p.u + (int64_t)p.perm[tile.row0 + min(16 * i + m, tile.nrows - 1)] * r + 32 * c + 8 * g;
#pragma unroll 4
      for (int s = 0; s < p.slices; ++s, ur += p.T * r) {
        u0 += *reinterpret_cast<const f32x4*>(ur);
        u1 += *reinterpret_cast<const f32x4*>(ur + 4);
      }
    }
    const Terms<TERMS> t = split<TERMS>(u0, u1);
#pragma unroll
    for (int h = 0; h < TERMS; ++h) us[w * TERMS + h][lane] = t.f[h];
  }
  // Every wave passes one barrier: with its first chunk on the way (T4096 N16384:
  // 79 us, 86 with the barrier first), or here without one.  Loads issued before u
  // would delay u, which waits for its own in the order of issue (12.5 -> 16 us
  // for 128 tokens of 64 adapters, N 16384).
  if (n_first >= N) lds_barrier();
  const uint16_t* const bb = p.b + (int64_t)tile.expert * p.N * r;
  for (int n = n_first; n < N; n += n_step) {
    uint4 y[MT][PIECES], bf[RC][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < PIECES; ++h)
        if (16 * i < tile.nrows) y[i][h] = load_y(i, h, n);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t at = (uint32_t)(min(n + col_of<BF16>(q, m), N - 1) * r + 8 * g);
#pragma unroll
      for (int c = 0; c < RC; ++c) {
        bf[c][q] = make_uint4(0, 0, 0, 0);
        if (32 * c + 8 * g < r) bf[c][q] = *reinterpret_cast<const uint4*>(bb + at + 32 * c);
      }
    }
    if (n == n_first) lds_barrier();
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (16 * i >= tile.nrows) break;
      f32x4 acc[4] = {};
#pragma unroll
      for (int c = 0; c < RC; ++c)
#pragma unroll
        for (int h = TERMS - 1; h >= 0; --h) {
          const uint4 u = us[(i * RC + c) * TERMS + h][lane];
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q] = mfma16(bf[c][q], u, acc[q]);
        }
      if (16 * i + m >= tile.nrows) continue;
#pragma unroll
      for (int h = 0; h < PIECES; ++h) {
        if (!inside(h, n)) continue;
        uint4 v;
        if constexpr (BF16)
          v = add_bf16(y[i][h], acc[2 * h], acc[2 * h + 1]);
        else
          v = __builtin_bit_cast(uint4, __builtin_bit_cast(f32x4, y[i][h]) + acc[h]);
        *reinterpret_cast<uint4*>(ob + row[i] + n * kSize + 64 * h) = v;
      }
    }
  }
}

template <bool BF16, int RC>
__global__ __launch_bounds__(64 * kUpWaves) void lora_up_few_kernel(LoraParams p) {
  lora_up<BF16, RC, kFewRows / 16>(p);
}
// Two waves per SIMD: each has 8 to 16 KiB of y on its way, and more of them only
// scatter the accesses (T4096 N16384 on changing inputs, waves per SIMD 1, 2, 3,
// 4: 110, 82, 83, 93 us).  The 16-token tiles want all the waves they can get
// (128 tokens of 64 adapters with 2, 3, 8: 27, 23, 18 us).
template <bool BF16, int RC>
__global__ __launch_bounds__(64 * kUpWaves) __attribute__((amdgpu_waves_per_eu(2, 2)))
void lora_up_kernel(LoraParams p) {
  lora_up<BF16, RC, kTileRows / 16>(p);
}

// out = y for the tokens without an adapter where the grouping does not list
// them (over kGroupTokens tokens; not needed in place).  row_bytes % 16 == 0.
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
  bool leader;
  size_t u, offsets, perm, tiles, ntiles, err, route, total;
  int tile_rows, max_tiles, slices;
};

Layout layout(int64_t T, int K, int r, int L) {
  Layout l;
  l.leader = T <= kLeaderTokens;
  // The ids are on the device, so the tile height follows the slots, as if each
  // had as many tokens as the others.  With few of many slots in use the short
  // tiles read an adapter more often than needed: 4096 tokens, N 16384, r 32, 8
  // adapters in 8 slots 89 us, in 512 slots 134; 16384 tokens, N 4096, one adapter
  // in 1 slot 116, in 512 slots 185.  Slices and column chunks count the tiles
  // that there may be, too: 256 tokens of one adapter (K 4096, N 16384, r 16) take
  // 36 us, of 64 adapters 26.
  l.tile_rows = l.leader || T <= 32 * (int64_t)L ? kFewRows : kTileRows;
  // the tokens without an adapter may add a tile
  l.max_tiles = l.leader ? (int)T : (int)((T + l.tile_rows - 1) / l.tile_rows + (T < L ? T : L) + 1);
  // Slices of K until there are a few workgroups per CU, four or more K steps
  // each.  The up kernel reads u once per slice, so a larger r gets fewer.
  if (l.tile_rows == kTileRows && K % 64 == 0)
    l.slices = std::max(1, std::min({512 / l.max_tiles, K / 64 / 4, r <= 64 ? 4 : 2}));
  else
    l.slices = std::max(1, std::min({512 / l.max_tiles, K / 128, r <= 64 ? 8 : 4}));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = up256(off + bytes);
    return at;
  };
  l.u = take(sizeof(float) * (size_t)l.slices * T * r);
  l.offsets = take(sizeof(int) * (size_t)(L + 1));
  l.perm = take(sizeof(int) * (size_t)T * (l.leader ? kFewRows : 1));
  l.tiles = take(sizeof(GemmTile) * (size_t)l.max_tiles);
  l.ntiles = take(sizeof(int));
  l.err = take(sizeof(int));
  l.route = take(T > kGroupTokens ? route_workspace_bytes(T, L) : 0);
  l.total = off;
  return l;
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int K, int r, int L) { return layout(T, K, r, L).total; }

hipError_t launch_lora_add(const void* y, bool bf16, int64_t T, int64_t N, const uint16_t* x, int K,
                           const uint16_t* a, const uint16_t* b, int r, int L, const int32_t* ids,
                           const float* scales, void* out, void* ws, hipStream_t s) {
  const Layout l = layout(T, K, r, L);
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
  p.slices = l.slices;
  p.tile_rows = l.tile_rows;
  p.tiles = reinterpret_cast<GemmTile*>(w + l.tiles);
  p.ntiles = l.leader ? nullptr : reinterpret_cast<int*>(w + l.ntiles);
  p.perm = reinterpret_cast<int*>(w + l.perm);
  p.u = reinterpret_cast<float*>(w + l.u);
  hipError_t e = hipSuccess;
  if (!l.leader) {
    if (T <= kGroupTokens) {
      lora_group_kernel<<<1, 1024, 0, s>>>(p);
      e = hipGetLastError();
    } else {
      e = launch_route(ids, T, L, l.tile_rows, 0, l.tile_rows, reinterpret_cast<int*>(w + l.offsets), p.perm, p.tiles,
                       p.ntiles, nullptr, nullptr, reinterpret_cast<int*>(w + l.err),
                       reinterpret_cast<int*>(w + l.route), nullptr, s);
    }
    if (e != hipSuccess) return e;
  }
  const int r16 = (r + 15) / 16, r32 = (r + 31) / 32;
  if (l.tile_rows == kFewRows || K % 64 != 0) {
    const dim3 grid((unsigned)l.slices, (unsigned)l.max_tiles, (unsigned)l.tile_rows / 16);
    auto go = [&](auto rt) {
      constexpr int RT = decltype(rt)::value;
      (l.leader ? lora_down_direct_kernel<RT, true>
                : lora_down_direct_kernel<RT, false>)<<<grid, 64 * kDirectWaves, 0, s>>>(p);
    };
    if (r16 == 1)
      go(std::integral_constant<int, 1>{});
    else if (r16 == 2)
      go(std::integral_constant<int, 2>{});
    else if (r16 <= 4)
      go(std::integral_constant<int, 4>{});
    else
      go(std::integral_constant<int, 8>{});
  } else {
    const dim3 grid((unsigned)l.slices, (unsigned)l.max_tiles);
    if (r32 == 1)
      lora_down_tile_kernel<1><<<grid, 256, 0, s>>>(p);
    else if (r32 == 2)
      lora_down_tile_kernel<2><<<grid, 256, 0, s>>>(p);
    else
      lora_down_tile_kernel<4><<<grid, 256, 0, s>>>(p);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  // a workgroup per 256 columns until there are enough of them
  const int64_t cols = (N + 64 * kUpWaves - 1) / (64 * kUpWaves);
  const int64_t per = std::max<int64_t>(1, std::min<int64_t>(cols, l.max_tiles * cols / 2048));
  const dim3 grid((unsigned)((cols + per - 1) / per), (unsigned)l.max_tiles);
  auto up = [&](auto rc) {
    constexpr int RC = decltype(rc)::value;
    if (l.tile_rows == kFewRows)
      (bf16 ? lora_up_few_kernel<true, RC> : lora_up_few_kernel<false, RC>)<<<grid, 64 * kUpWaves, 0, s>>>(p);
    else
      (bf16 ? lora_up_kernel<true, RC> : lora_up_kernel<false, RC>)<<<grid, 64 * kUpWaves, 0, s>>>(p);
  };
  if (r32 == 1)
    up(std::integral_constant<int, 1>{});
  else if (r32 == 2)
    up(std::integral_constant<int, 2>{});
  else if (r32 == 3)
    up(std::integral_constant<int, 3>{});
  else
    up(std::integral_constant<int, 4>{});
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (T > kGroupTokens && out != y) lora_copy_kernel<<<(unsigned)T, 256, 0, s>>>(p, N * (bf16 ? 2 : 4));
  return hipGetLastError();
}

}  // namespace nvfp4
