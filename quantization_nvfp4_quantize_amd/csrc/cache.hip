// A cache whose rows are quantized as they are written and dequantized as they
// are read: NVFP4 and MXFP4 rows (the bytes of the tensor quantizers) and
// MXFP8 rows (32 E4M3 elements per E8M0 scale, OCP MX v1.0).
//
// A slot holds one row of R elements (all heads of one token); rows are
// independent, so writing one never touches what another holds.  Writes are cut
// into chunks of 8 elements: a lane loads 16 bytes of bf16, the 2 (NVFP4) or 4
// (MX) lanes of a block exchange their maxima with DPP, and a block never
// straddles two rows because R is a multiple of its length.  Both directions are
// bound by memory: writing MXFP8 (T16384, keys and values) moves 5.9 TB/s, reading
// 24 sequences 6.0 with the cache's bytes partly in the memory-side cache and 4.9
// without, what a copy of 2 + 2 GiB moves; with streaming stores for what the
// call does not read again.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "launch.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kCacheThreads = 256;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// i / d for i < 2^31, d >= 1, as one high product, an add and a shift.
struct FastDiv {
  uint32_t mul, shift;
};

FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  return {(uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1), l};
}

__device__ __forceinline__ uint32_t divide(uint32_t i, FastDiv f) { return (__umulhi(i, f.mul) + i) >> f.shift; }

struct PartParams {
  const uint16_t* x;  // write: the rows
  int64_t stride;     // write: elements from one row to the next
  void* out;          // read: [T][R]
  uint8_t* q;
  uint8_t* s;
  const float* gs;
  uint32_t r8;        // chunks per row
  uint32_t n8;        // chunks in all
  FastDiv by_r8;
};

struct CacheParams {
  PartParams part[2];
  const int32_t* slots;  // nullable: by page table
  uint32_t n_slots;
  const int32_t* pages;    // [B][wide]
  const int32_t* cu_lens;  // [B + 1]
  int B, wide, page_size;
};

// Maximum over the 4 lanes of a quad.
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, false)));
  return fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, false)));
}

// E8M0 code of an MXFP4 block with largest magnitude m: floor(log2(m)) - 2 + 127
// from m's exponent bits, clamped at 0 (as mxfp4_quantize).
__device__ __forceinline__ uint32_t mx4_code(float m) { return (uint32_t)max((int)(__float_as_uint(m) >> 23) - 2, 0); }

// E8M0 code of an MXFP8 block: the smallest scale at which nothing saturates,
// m <= 448 * 2^(code - 127).  448 = 1.75 * 2^8, so that is floor(log2(m)) - 8,
// and one more for a significand above 1.75 (upper seven bits above 0x60;
// the rest of a bf16 value is 0).
__device__ __forceinline__ uint32_t mx8_code(float m) {
  const uint32_t b = __float_as_uint(m);
  return (uint32_t)max((int)(b >> 23) - 8 + (int)((b & 0x7fffffu) > 0x600000u), 0);
}

template <int FMT, int UNROLL>
__global__ __launch_bounds__(kCacheThreads) void cache_write_kernel(CacheParams p) {
  constexpr int kChunks = kCacheThreads * UNROLL;
  __shared__ float rtab[FMT == kNvfp4 ? 128 : 1];
  const PartParams c = blockIdx.y ? p.part[1] : p.part[0];
  const uint32_t base = blockIdx.x * kChunks + threadIdx.x;
  if (blockIdx.x * (uint32_t)kChunks >= c.n8) return;  // the other part has longer rows
  uint4 w[UNROLL];
  uint32_t slot[UNROLL], col[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t i = base + u * kCacheThreads;
    slot[u] = ~0u;
    col[u] = 0;
    w[u] = make_uint4(0, 0, 0, 0);
    if (i < c.n8) {
      const uint32_t row = divide(i, c.by_r8);
      col[u] = i - row * c.r8;
      slot[u] = (uint32_t)p.slots[row];
      w[u] = *reinterpret_cast<const uint4*>(c.x + (int64_t)row * c.stride + 8 * (int64_t)col[u]);
    }
  }
  float E = 0.0f;
  if constexpr (FMT == kNvfp4) {
    E = 1.0f / c.gs[0];
    fill_rtab(rtab, E, threadIdx.x);
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const bool on = slot[u] < p.n_slots;  // also false for -1
    const int64_t at = (int64_t)slot[u] * c.r8 + col[u];
    if constexpr (FMT == kNvfp4) {
      uint32_t sf;
      const uint32_t n = quantize_half_block(w[u], E, rtab, &sf);
      if (on) {
        __builtin_nontemporal_store(n, reinterpret_cast<uint32_t*>(c.q) + at);
        if ((col[u] & 1) == 0) c.s[at >> 1] = (uint8_t)sf;
      }
    } else {
      const float m = quad_max(abs_max8(w[u]));
      const uint32_t code = FMT == kMxfp4 ? mx4_code(m) : mx8_code(m);
      const float r = __uint_as_float((254u - code) << 23);  // 2^(127 - code), exact
      const uint32_t d[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      if constexpr (FMT == kMxfp4) {
        uint32_t n = 0;
        n = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(n, bf16_lo(d[0]) * r, bf16_hi(d[0]) * r, 1.0f, 0);
        n = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(n, bf16_lo(d[1]) * r, bf16_hi(d[1]) * r, 1.0f, 1);
        n = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(n, bf16_lo(d[2]) * r, bf16_hi(d[2]) * r, 1.0f, 2);
        n = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(n, bf16_lo(d[3]) * r, bf16_hi(d[3]) * r, 1.0f, 3);
        if (on) __builtin_nontemporal_store(n, reinterpret_cast<uint32_t*>(c.q) + at);
      } else {
        u32x2 e;  // |x * r| <= 448: the conversion rounds to nearest even there
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int v = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(d[2 * h]) * r, bf16_hi(d[2 * h]) * r, 0, false);
          e[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(d[2 * h + 1]) * r, bf16_hi(d[2 * h + 1]) * r, v,
                                                           true);
        }
        if (on) __builtin_nontemporal_store(e, reinterpret_cast<u32x2*>(c.q) + at);
      }
      if (on && (col[u] & 3) == 0) c.s[at >> 2] = (uint8_t)code;
    }
  }
}

// Elements 2 h and 2 h + 1 of a dword of E2M1 nibbles, or of half a dword of E4M3 bytes.
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f32x2 pair_fp4(uint32_t q, int h) {
  return h == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0)
         : h == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1)
         : h == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2)
                  : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
}
__device__ __forceinline__ f32x2 pair_fp8(uint32_t q, int h) {
  return h ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, 1.0f, false);
}

constexpr float kLargestBf16 = 0x1.fep127f;
constexpr uint32_t kZeros = 0xffffffffu;  // the row is read as zeros
constexpr uint32_t kSkip = 0xfffffffeu;   // the row belongs to no sequence and is left as it was

// The slot of output row t by page table: the sequence b with cu_lens[b] <= t
// < cu_lens[b + 1], then its page.  Every index is checked before it is used.
__device__ __forceinline__ uint32_t slot_of_row(const CacheParams& p, uint32_t t) {
  int lo = 0, hi = p.B;  // the first b with cu_lens[b + 1] > t
  while (lo < hi) {
    const int mid = lo + ((hi - lo) >> 1);  // lo + hi may pass 2^31
    if (p.cu_lens[mid + 1] > (int64_t)t) hi = mid;
    else lo = mid + 1;
  }
  if (lo >= p.B) return kSkip;
  const int64_t pos = (int64_t)t - p.cu_lens[lo];
  if (pos < 0) return kSkip;
  const uint32_t page = (uint32_t)pos / (uint32_t)p.page_size;
  if (page >= (uint32_t)p.wide) return kZeros;
  const int32_t id = p.pages[(int64_t)lo * p.wide + page];
  if (id < 0) return kZeros;
  const int64_t slot = (int64_t)id * p.page_size + ((uint32_t)pos - page * (uint32_t)p.page_size);
  return slot < p.n_slots ? (uint32_t)slot : kZeros;
}

// A workgroup's units belong to a few consecutive rows: one thread per row finds
// its slot (a search in cu_lens, a load from the page table), all read it from
// LDS.  A unit is what 16 bytes of output hold, 8 bf16 or 4 fp32 elements, so
// that a store instruction of a wave fills whole lines; then non-temporal
// stores pay (24 sequences of up to 8192 rows of 576 into bf16: 28.7 us against
// 39.7; two of them 32 bytes apart per lane into fp32: 95 against 64).
template <int FMT, bool BF16_OUT, int UNROLL>
__global__ __launch_bounds__(kCacheThreads) void cache_read_kernel(CacheParams p) {
  constexpr int kUnit = BF16_OUT ? 8 : 4, kUnits = kCacheThreads * UNROLL, kPerBlock = (FMT == kNvfp4 ? 16 : 32) / kUnit;
  __shared__ uint32_t slots[kUnits * kUnit / 16 + 2];  // a row has 16 elements at least
  const PartParams c = blockIdx.y ? p.part[1] : p.part[0];
  const uint32_t per_row = c.r8 * (8 / kUnit), n = c.n8 * (8 / kUnit), first = blockIdx.x * (uint32_t)kUnits;
  if (first >= n) return;
  const uint32_t last = min(first + (uint32_t)kUnits, n) - 1;
  const auto row_of = [&](uint32_t i) { return divide(i / (8 / kUnit), c.by_r8); };
  const uint32_t row0 = row_of(first), rows = row_of(last) - row0 + 1;
  for (uint32_t r = threadIdx.x; r < rows; r += kCacheThreads) {
    uint32_t s;
    if (p.slots) {
      s = (uint32_t)p.slots[row0 + r];
      if (s >= p.n_slots) s = kZeros;
    } else {
      s = slot_of_row(p, row0 + r);
    }
    slots[r] = s;
  }
  const float g = FMT == kNvfp4 ? c.gs[0] : 1.0f;
  __syncthreads();
  uint32_t slot[UNROLL], code[UNROLL];
  u32x2 q[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t i = first + threadIdx.x + u * kCacheThreads;
    slot[u] = kSkip;
    code[u] = 0;
    q[u] = u32x2{0, 0};
    if (i < n) {
      const uint32_t row = row_of(i), col = i - row * per_row;
      slot[u] = slots[row - row0];
      if (slot[u] < kSkip) {
        const int64_t at = (int64_t)slot[u] * per_row + col;
        code[u] = c.s[at / kPerBlock];
        if constexpr (FMT == kMxfp8 && BF16_OUT) q[u] = reinterpret_cast<const u32x2*>(c.q)[at];
        else if constexpr (FMT == kMxfp8 || BF16_OUT) q[u][0] = reinterpret_cast<const uint32_t*>(c.q)[at];
        else q[u][0] = reinterpret_cast<const uint16_t*>(c.q)[at];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    if (slot[u] == kSkip) continue;
    float v[kUnit];
#pragma unroll
    for (int h = 0; h < kUnit / 2; ++h) {
      const auto e = FMT == kMxfp8 ? pair_fp8(q[u][h / 2], h & 1) : pair_fp4(q[u][0], h);
      v[2 * h] = e[0];
      v[2 * h + 1] = e[1];
    }
    if constexpr (FMT == kNvfp4) {
      const float sfd = e4m3_decode_signed(code[u]);
#pragma unroll
      for (int k = 0; k < kUnit; ++k) v[k] = (v[k] * sfd) * g;
    } else {
      const int e = (int)code[u] - 127;
#pragma unroll
      for (int k = 0; k < kUnit; ++k) v[k] = ldexpf(v[k], e);
      // Blocks with a maximum above 1.75 * 2^127 have code 247, and elements from
      // 1.9375 * 2^127 on are rounded up to 2^128 there.  They stand for bf16
      // values, so they are read as the largest of these.  (NaN stays.)
      if (FMT == kMxfp8 && code[u] >= 247) {
#pragma unroll
        for (int k = 0; k < kUnit; ++k)
          if (isinf(v[k])) v[k] = copysignf(kLargestBf16, v[k]);
      }
    }
    u32x4 o;
    if constexpr (BF16_OUT) {
      __bf16 h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] = (__bf16)v[k];
      __builtin_memcpy(&o, h, 16);
    } else {
      __builtin_memcpy(&o, v, 16);
    }
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(c.out) + ((int64_t)first + threadIdx.x + u * kCacheThreads));
  }
}

CacheParams params_of(const CachePart* parts, int n, int64_t T) {
  CacheParams p = {};
  for (int i = 0; i < n; ++i) {
    const CachePart& s = parts[i];
    const uint32_t r8 = (uint32_t)(s.R / 8);
    p.part[i] = {s.x, s.x_stride, s.out, s.q, s.s, s.gs, r8, (uint32_t)(T * r8), fast_div(r8)};
  }
  return p;
}

// Grid for units of `elements` elements, `per` of them per workgroup.
dim3 grid_of(const CacheParams& p, int n, uint32_t elements, uint32_t per) {
  const uint32_t most = std::max(p.part[0].n8, n > 1 ? p.part[1].n8 : 0u) * (8 / elements);
  return dim3((most + per - 1) / per, n);
}

template <int FMT, bool BF16_OUT, int UNROLL>
void read_with(const CacheParams& p, int n, hipStream_t s) {
  const dim3 g = grid_of(p, n, BF16_OUT ? 8 : 4, kCacheThreads * UNROLL);
  cache_read_kernel<FMT, BF16_OUT, UNROLL><<<g, kCacheThreads, 0, s>>>(p);
}

// Four units per thread keep enough loads in flight for large reads (24 sequences
// of up to 8192 rows of 576: 28.5 us against 38.6 with one, 29.6 with two); where
// that leaves CUs without a workgroup, one (262 rows of 8 x 128, keys and values: 3.35 us against 4.1).
// Rows of 576 by slot into bf16, one unit against four (us, NVFP4 and MXFP8), at
// workgroups of four units: 120 2.60 and 3.33, 2.58 and 3.36; 250 2.97 and 3.53,
// 3.01 and 3.52; 500 3.38 and 3.74, 3.64 and 4.02; 700 4.36 and 4.26, 4.85 and 4.51;
// 2000 9.44 and 9.36, 10.61 and 10.10.  One would do better up to some 600; the
// bound stands where every CU has work.
template <int FMT, bool BF16_OUT>
void read_as(const CacheParams& p, int n, hipStream_t s) {
  const dim3 g = grid_of(p, n, BF16_OUT ? 8 : 4, 4 * kCacheThreads);
  if (g.x * g.y <= 256) read_with<FMT, BF16_OUT, 1>(p, n, s);
  else read_with<FMT, BF16_OUT, 4>(p, n, s);
}

template <int FMT>
hipError_t read_format(const CacheParams& p, int n, bool bf16_out, hipStream_t s) {
  if (bf16_out) read_as<FMT, true>(p, n, s);
  else read_as<FMT, false>(p, n, s);
  return hipGetLastError();
}

hipError_t launch_read(int fmt, const CacheParams& p, int n, bool bf16_out, hipStream_t s) {
  if (fmt == kNvfp4) return read_format<kNvfp4>(p, n, bf16_out, s);
  if (fmt == kMxfp4) return read_format<kMxfp4>(p, n, bf16_out, s);
  return read_format<kMxfp8>(p, n, bf16_out, s);
}

// Two chunks per thread: T16384, keys and values of 8 x 128 into MXFP8 17.1 us
// (5.9 TB/s) against 17.9 with one or four.
template <int FMT>
hipError_t write_format(const CacheParams& p, int n, hipStream_t s) {
  cache_write_kernel<FMT, 2><<<grid_of(p, n, 8, 2 * kCacheThreads), kCacheThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(int fmt, const CachePart* parts, int n, int64_t T, const int32_t* slots, int64_t n_slots,
                              hipStream_t s) {
  if (T == 0) return hipSuccess;
  CacheParams p = params_of(parts, n, T);
  p.slots = slots;
  p.n_slots = (uint32_t)n_slots;
  if (fmt == kNvfp4) return write_format<kNvfp4>(p, n, s);
  if (fmt == kMxfp4) return write_format<kMxfp4>(p, n, s);
  return write_format<kMxfp8>(p, n, s);
}

hipError_t launch_cache_read(int fmt, const CachePart* parts, int n, int64_t T, const int32_t* slots, int64_t n_slots,
                             bool bf16_out, hipStream_t s) {
  if (T == 0) return hipSuccess;
  CacheParams p = params_of(parts, n, T);
  p.slots = slots;
  p.n_slots = (uint32_t)n_slots;
  return launch_read(fmt, p, n, bf16_out, s);
}

hipError_t launch_cache_read_pages(int fmt, const CachePart* parts, int n, int64_t T, const int32_t* pages, int64_t B,
                                   int64_t wide, int64_t page_size, const int32_t* cu_lens, int64_t n_slots,
                                   bool bf16_out, hipStream_t s) {
  if (T == 0 || B == 0) return hipSuccess;
  CacheParams p = params_of(parts, n, T);
  p.pages = pages;
  p.cu_lens = cu_lens;
  p.B = (int)B;
  p.wide = (int)wide;
  p.page_size = (int)page_size;
  p.n_slots = (uint32_t)n_slots;
  return launch_read(fmt, p, n, bf16_out, s);
}

}  // namespace nvfp4
