// The 8-bit paged latent KV cache: appending tokens to it and reading them back.
//
// The cache holds e4m3 codes [pages, page_size, 576] with one fp32 scale per page (a page
// is the block of tokens that shares a scale; MLA has one KV head); a value is code * scale.
// The scale is the smallest power of two s with amax <= 448 s, amax over the page's finite
// entries, so dividing by it is exact and a page whose scale grows by 2^k only has 2^k
// taken off its codes' exponents: they stay exact down to e4m3's subnormals, where they are
// rounded once more. 448 = 1.75 * 2^8 makes the scale's exponent that of amax minus 8, plus
// one if amax's significand exceeds 1.75.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace fp8moe {

constexpr int kLatDk = 576;                  // entries of a cache row (512 latent + 64 rotary)
constexpr int kLatVec = kLatDk / 8;          // 16-byte pieces of a bf16 row
constexpr int kScaleMinExp = -110;           // keeps 1 / scale and products with it normal fp32

// These kernels and the attention's are launched while the work before them may still write what they read
// (a page's scale, say, that the append before a decode has just raised), and wait for its end themselves.
// A kernel's whole life counts for the read-only path (__ldg, ld.global.nc), the time before that wait too,
// and a line that an SM read over it earlier may be an old one. So all their loads are ordinary ones.

// The page table of a batch, and the buffer it points into.
struct PageTable {
  const int32_t* indptr;         // [B + 1]
  const int32_t* indices;        // [num_indices]
  const int32_t* last_lens;      // [B]
  int B, num_pages, page_size, num_indices;
};

// First page-table entry and token count of sequence b; false (and flagged) if the table's
// entries for it are out of range. An empty sequence is a valid one of 0 tokens.
__device__ __forceinline__ bool sequence_extent(const PageTable& t, int b, int& first, int& len) {
  const int lo = t.indptr[b], hi = t.indptr[b + 1], last = t.last_lens[b];
  first = lo;
  len = 0;
  if (lo < 0 || hi < lo || hi > t.num_indices) {
    raise_device_error(FP8MOE_DEVERR_PAGE);
    return false;
  }
  if (hi == lo) return true;
  if (last < 1 || last > t.page_size) {
    raise_device_error(FP8MOE_DEVERR_PAGE);
    return false;
  }
  len = (hi - lo - 1) * t.page_size + last;
  return true;
}

// The page at entry `at` of the table (already known to be below num_indices); -1 and flagged
// if it lies outside the buffer.
__device__ __forceinline__ int table_page(const PageTable& t, int at) {
  const int page = t.indices[at];
  if (page < 0 || page >= t.num_pages) {
    raise_device_error(FP8MOE_DEVERR_PAGE);
    return -1;
  }
  return page;
}

// Four e4m3 codes <-> fp32.
__device__ __forceinline__ float4 e4m3x4_to_float(uint32_t codes) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ uint32_t float_to_e4m3x4(float a, float b, float c, float d) {
  return static_cast<uint32_t>(cvt_e4m3x2(a, b)) | (static_cast<uint32_t>(cvt_e4m3x2(c, d)) << 16);
}
__device__ __forceinline__ float2 bf16x2_to_float(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// Whether a sequence's range lo .. hi - 1 lies within `rows` rows.
__device__ __forceinline__ bool range_fits(int lo, int hi, int rows) { return lo >= 0 && hi >= lo && hi <= rows; }

// Products and quotients under a caller's scale that is no power of two. fp32 would round them before the code
// or bf16 value does, now and then onto the middle of two of those; here the neighbour with an odd last
// bit stands for what lies between two fp32 values, so that the later rounding is as good as the only one.
__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }
__device__ __forceinline__ float odd_of(float down, float up) {
  return down == up || (__float_as_uint(down) & 1u) ? down : up;
}
__device__ __forceinline__ float product_to_odd(float x, float s) { return odd_of(__fmul_rd(x, s), __fmul_ru(x, s)); }
__device__ __forceinline__ float quotient_to_odd(float x, float s) { return odd_of(__fdiv_rd(x, s), __fdiv_ru(x, s)); }

// ---------------------------------------------------------------- append
struct AppendArgs {
  const __nv_bfloat16* kv_new;   // [T, 576], row stride ld
  long long ld;
  const int32_t* append_indptr;  // [B + 1]
  uint8_t* cache;
  float* scale;                  // [num_pages]
  PageTable table;
  int T;
};

constexpr int kAppendHeld = 8;  // rows a thread keeps its 16 bytes of in registers between the passes
constexpr int kAppendMaxRows = 7;   // rows a CTA handles side by side: 7 * 72 = 504 threads

// Two bf16 magnitudes' bit patterns, non-finite ones as 0 (their order is that of the values).
__device__ __forceinline__ uint32_t finite_magnitudes(uint32_t v) {
  v &= 0x7fff7fffu;
  return v & ~__vcmpgeu2(v, 0x7f807f80u);
}

// Sequences that start by some place, which grows with b: all threads of the CTA search together, one
// round where there are no more sequences than threads, three (256 threads) or four (96) for the 2^20 there can be.
template <typename F>
__device__ __forceinline__ int count_sequences(int B, F&& starts_by) {
  const int threads = static_cast<int>(blockDim.x);
  int lo = 0, hi = B;                                        // the count lies between them
  while (lo < hi) {
    const int step = hi - lo <= threads ? 1 : (hi - lo + threads - 1) / threads;
    const int at = lo + (static_cast<int>(threadIdx.x) + 1) * step - 1;     // the last of this thread's share
    lo += __syncthreads_count(at < hi && starts_by(at)) * step;
    hi = min(hi, lo + step - 1);
  }
  return hi;
}

// A thread's 8 columns of every `side`-th of `rows` rows, under a scale that is no power of two.
__device__ __noinline__ void append_under_any_scale(const __nv_bfloat16* src, long long ld, uint8_t* dst, int rows, int side,
                                                    float s) {
  for (int r = 0; r < rows; r += side) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const float x = __bfloat162float(src[r * ld + i]);
      dst[static_cast<size_t>(r) * kLatDk + i] = static_cast<uint8_t>(cvt_e4m3x2(quotient_to_odd(x, s), 0.0f));
    }
  }
}

// One CTA per (sequence, page written): the largest magnitude of the page's new rows, the page's
// scale, the codes. Sequence b owns the CTAs from floor(append_indptr[b] / page_size) + 2b on:
// its n tokens touch at most floor(n / page_size) + 2 pages, and the floors leave room for that.
// A thread owns one 16-byte column of every `side`-th row. The rows are read once (held in
// registers up to 8 each, read again beyond), before the page itself is looked up. Bound by the
// chain of dependent loads at decode and prompt sizes (four of them: one token for 64 sequences 2.8 us, 4096
// tokens 5.5), by HBM beyond (16K tokens in pages of 16 9.9 us).
__global__ void __launch_bounds__(512, 2) mla_kv_append_kernel(const AppendArgs a, int side) {
  __shared__ uint32_t warp_max[16];
  const int tid = threadIdx.x;
  const int ps = a.table.page_size;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the work before this in the stream is done
  // Every range is looked at by some thread (there are at least twice as many blocks as sequences): one that
  // decreases may have no block, the next sequence's having taken its place.
  const long long looked = static_cast<long long>(blockIdx.x) * blockDim.x + tid;
  int2 range = make_int2(0, 0);
  if (looked < a.table.B) range = make_int2(a.append_indptr[looked], a.append_indptr[looked + 1]);
  const int count = count_sequences(
      a.table.B, [&](int b) { return a.append_indptr[b] / ps + 2ll * b <= blockIdx.x; });
  if (!range_fits(range.x, range.y, a.T)) raise_device_error(FP8MOE_DEVERR_PAGE);
  if (count == 0) return;
  const int b = count - 1;
  const int lo = a.append_indptr[b], hi = a.append_indptr[b + 1];
  int first, len;
  const bool table = sequence_extent(a.table, b, first, len);
  const long long nth = blockIdx.x - (lo / ps + 2ll * b);    // negative only where the ranges decrease
  if (!range_fits(lo, hi, a.T) || nth < 0 || (table && hi - lo > len)) {
    if (tid == 0) raise_device_error(FP8MOE_DEVERR_PAGE);
    return;
  }
  if (!table || hi == lo) return;
  const int start = len - (hi - lo);                         // position of the first new token
  if (start / ps + nth > (len - 1) / ps) return;
  const int j = start / ps + static_cast<int>(nth);
  const int pos0 = max(start, j * ps);                       // (j * ps <= len - 1: no overflow)
  const int slot0 = pos0 - j * ps;
  const int rows = static_cast<int>(min(static_cast<long long>(len), (j + 1ll) * ps) - pos0);
  const int r0 = tid / kLatVec, col = tid - r0 * kLatVec;
  const bool active = r0 < side;
  const __nv_bfloat16* src = a.kv_new + (lo + (pos0 - start) + static_cast<long long>(r0)) * a.ld + col * 8;
  const long long step = static_cast<long long>(side) * a.ld;
  uint4 held[kAppendHeld];
  uint32_t mx = 0;
  auto take = [&](const uint4& x) {
    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(finite_magnitudes(x.x), finite_magnitudes(x.y)),
                               __vmaxu2(finite_magnitudes(x.z), finite_magnitudes(x.w))));
  };
#pragma unroll
  for (int i = 0; i < kAppendHeld; ++i)
    held[i] = active && r0 + i * side < rows ? *reinterpret_cast<const uint4*>(src + i * step) : make_uint4(0, 0, 0, 0);
  const int page = table_page(a.table, first + j);
  if (page < 0) return;                                      // (the same for the whole CTA)
  const float old = slot0 > 0 ? a.scale[page] : 0.0f;        // a page written from its first slot starts afresh
#pragma unroll
  for (int i = 0; i < kAppendHeld; ++i) take(held[i]);
  if (active)
    for (int r = r0 + kAppendHeld * side; r < rows; r += side)
      take(*reinterpret_cast<const uint4*>(src + static_cast<long long>(r - r0) * a.ld));
  mx = max(mx & 0xffffu, mx >> 16);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((tid & 31) == 0) warp_max[tid >> 5] = mx;
  __syncthreads();
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) mx = max(mx, warp_max[w]);

  float s = 0.0f;
  if (mx != 0) {
    const int ex = max(kScaleMinExp, static_cast<int>(mx >> 7) - 135 + ((mx & 0x7fu) > 96u ? 1 : 0));
    s = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
  }
  s = fmaxf(s, old);
  if (tid == 0) a.scale[page] = s;                           // every thread read `old` before the barrier
  const float inv = s > 0.0f ? 1.0f / s : 1.0f;
  uint8_t* page_codes = a.cache + static_cast<size_t>(page) * ps * kLatDk;
  uint8_t* dst = page_codes + static_cast<size_t>(slot0 + r0) * kLatDk + col * 8;
  auto store = [&](int r, const uint4& x) {                  // r rows below this thread's first
    const float2 f0 = bf16x2_to_float(x.x), f1 = bf16x2_to_float(x.y), f2 = bf16x2_to_float(x.z),
                 f3 = bf16x2_to_float(x.w);
    *reinterpret_cast<uint2*>(dst + static_cast<size_t>(r) * kLatDk) =
        make_uint2(float_to_e4m3x4(f0.x * inv, f0.y * inv, f1.x * inv, f1.y * inv),
                   float_to_e4m3x4(f2.x * inv, f2.y * inv, f3.x * inv, f3.y * inv));
  };
  if (power_of_two(s)) {
#pragma unroll
    for (int i = 0; i < kAppendHeld; ++i)
      if (active && r0 + i * side < rows) store(i * side, held[i]);
    if (active)
      for (int r = r0 + kAppendHeld * side; r < rows; r += side)
        store(r - r0, *reinterpret_cast<const uint4*>(src + static_cast<long long>(r - r0) * a.ld));
  } else if (active) {
    append_under_any_scale(src, a.ld, dst, rows - r0, side, s);
  }

  // the rows that were there, in the larger scale (from a scale of 0, under which any code stands for 0, as codes of 0)
  if (slot0 > 0 && s > old) {
    const float ratio = old / s;
    uint4* codes = reinterpret_cast<uint4*>(page_codes);
    for (long long v = tid; v < static_cast<long long>(slot0) * (kLatDk / 16); v += blockDim.x) {
      uint4 x = codes[v];
      uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = e4m3x4_to_float(w[i]);
        w[i] = power_of_two(old) ? float_to_e4m3x4(f.x * ratio, f.y * ratio, f.z * ratio, f.w * ratio)
                                 : float_to_e4m3x4(product_to_odd(f.x, ratio), product_to_odd(f.y, ratio),
                                                   product_to_odd(f.z, ratio), product_to_odd(f.w, ratio));
      }
      codes[v] = x;
    }
  }
}

// ---------------------------------------------------------------- gather
struct GatherArgs {
  const uint8_t* cache;
  const float* scale;
  PageTable table;
  const int32_t* out_indptr;     // [B + 1]
  __nv_bfloat16* out;            // [T, 576], row stride ld
  long long ld;
  int T;
  bool wide;                     // every output row begins at a multiple of 32 bytes
};

constexpr int kGatherRows = 32;
constexpr int kGatherThreads = 256;

// 16 codes under a scale that is no power of two (out of line: in the loop below it cost short prefixes 0.5 us).
__device__ __noinline__ void gather_under_any_scale(const uint4 codes, float s, __nv_bfloat16* dst) {
  uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll 1
  for (int i = 0; i < 4; ++i, dst += 4) {
    const float4 f = e4m3x4_to_float(w[0]);
    w[0] = w[1];
    w[1] = w[2];
    w[2] = w[3];
    dst[0] = __float2bfloat16_rn(product_to_odd(f.x, s));
    dst[1] = __float2bfloat16_rn(product_to_odd(f.y, s));
    dst[2] = __float2bfloat16_rn(product_to_odd(f.z, s));
    dst[3] = __float2bfloat16_rn(product_to_odd(f.w, s));
  }
}

// A CTA reads back 32 output rows: their cache rows first (a thread each), then 16 codes at a
// time (one 16-byte load, one 32-byte store). Bound by HBM, of whose bytes two thirds are written (32 prefixes of
// 4096: 34.3 us, 0.90 of it).
__global__ void __launch_bounds__(kGatherThreads) mla_kv_gather_kernel(const GatherArgs a) {
  __shared__ long long row_at[kGatherRows];                  // cache row, or -1
  __shared__ float row_scale[kGatherRows];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * kGatherRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the work before this in the stream is done
  // Every range is looked at by some thread, the ones without a row here too (asked for before the search, as
  // both wait for memory).
  const int looked = blockIdx.x * kGatherThreads + tid;
  int2 range = make_int2(0, 0);
  if (looked < a.table.B) range = make_int2(a.out_indptr[looked], a.out_indptr[looked + 1]);
  const int before = count_sequences(a.table.B, [&](int b) { return a.out_indptr[b] <= t0; });
  if (!range_fits(range.x, range.y, a.T)) raise_device_error(FP8MOE_DEVERR_PAGE);
  if (t0 >= a.T) return;
  if (tid < kGatherRows) {
    const int t = t0 + tid;
    long long at = -1;
    float sc = 0.0f;
    int b = max(before - 1, 0);
    while (b < a.table.B && a.out_indptr[b + 1] <= t) ++b;
    if (t < a.T && b < a.table.B) {
      const int lo = a.out_indptr[b];
      int first, len;
      if (t >= lo && range_fits(lo, a.out_indptr[b + 1], a.T) && sequence_extent(a.table, b, first, len)) {
        const int i = t - lo;
        if (i >= len) {
          raise_device_error(FP8MOE_DEVERR_PAGE);
        } else {
          const int page = table_page(a.table, first + i / a.table.page_size);
          if (page >= 0) {
            at = static_cast<long long>(page) * a.table.page_size + i % a.table.page_size;
            sc = a.scale[page];
          }
        }
      }
    }
    row_at[tid] = at;
    row_scale[tid] = sc;
  }
  __syncthreads();
  constexpr int kPieces = kLatDk / 16, kMine = (kGatherRows * kPieces + kGatherThreads - 1) / kGatherThreads;
  uint4 codes[kMine];                                        // all loads before the first store
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int v = tid + i * kGatherThreads, r = v / kPieces;
    if (v < kGatherRows * kPieces && row_at[r] >= 0)
      codes[i] = reinterpret_cast<const uint4*>(a.cache + row_at[r] * kLatDk)[v - r * kPieces];
  }
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int v = tid + j * kGatherThreads, r = v / kPieces, c = v - r * kPieces;
    if (v >= kGatherRows * kPieces || row_at[r] < 0) continue;
    const float s = row_scale[r];
    const uint4 x = codes[j];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    __align__(16) __nv_bfloat162 y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = e4m3x4_to_float(w[i]);
      y[2 * i] = __floats2bfloat162_rn(f.x * s, f.y * s);
      y[2 * i + 1] = __floats2bfloat162_rn(f.z * s, f.w * s);
    }
    uint4* dst = reinterpret_cast<uint4*>(a.out + (t0 + r) * a.ld) + 2 * c;
    if (!power_of_two(s)) {
      gather_under_any_scale(x, s, reinterpret_cast<__nv_bfloat16*>(dst));
    } else if (a.wide) {
      st_global_v8(dst, reinterpret_cast<const uint32_t(&)[8]>(y));
    } else {
      dst[0] = *reinterpret_cast<const uint4*>(&y[0]);
      dst[1] = *reinterpret_cast<const uint4*>(&y[4]);
    }
  }
}

}  // namespace fp8moe
