// Multi-head latent attention over the 8-bit paged latent cache: one warp per (query token, head).
//
// s_j = sm_scale <q, k_j> over 576 entries (soft-capped if asked), o = softmax(s) V with V the
// first 512 entries of the same rows. Online softmax in base 2, everything in fp32.
#pragma once

#include "mla_fp8_cache.cuh"

namespace fp8moe {

constexpr int kLatDv = 512;

struct LatAttnArgs {
  const __nv_bfloat16* q;        // [num_q, Hq, 576]
  const int32_t* qo_indptr;      // [B + 1], or null: one query token per sequence
  const uint8_t* cache;
  const float* scale;
  PageTable table;
  __nv_bfloat16* o;              // [num_q, Hq, 512]
  float* lse;                    // [num_q, Hq] or null
  int num_q, Hq;
  float sm_scale, logit_cap;
};

__global__ void __launch_bounds__(128) mla_fp8_simple_kernel(const LatAttnArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y * 4 + warp, t = blockIdx.x;
  if (h >= a.Hq) return;
  int b = t, n = 1, i = 0;
  if (a.qo_indptr) {
    b = 0;
    while (b < a.table.B && __ldg(a.qo_indptr + b + 1) <= t) ++b;
    if (b == a.table.B) return;
    const int lo = __ldg(a.qo_indptr + b), hi = __ldg(a.qo_indptr + b + 1);
    if (t < lo) return;
    if (lo < 0 || hi > a.num_q) {
      raise_device_error(FP8MOE_DEVERR_PAGE);
      return;
    }
    n = hi - lo;
    i = t - lo;
  }
  int first, len;
  if (!sequence_extent(a.table, b, first, len)) len = 0;
  const int sees = min(len, max(0, len - n + i + 1));
  const size_t row = static_cast<size_t>(t) * a.Hq + h;
  float q[20], acc[16];
  for (int k = 0; k < 16; ++k) {
    q[k] = __bfloat162float(a.q[row * kLatDk + lane * 16 + k]);
    acc[k] = 0.0f;
  }
  q[16] = __bfloat162float(a.q[row * kLatDk + 512 + 2 * lane]);
  q[17] = __bfloat162float(a.q[row * kLatDk + 513 + 2 * lane]);
  const float kLog2e = 1.4426950408889634f;
  float m = -INFINITY, l = 0.0f;
  for (int j = 0; j < sees; ++j) {
    int page = table_page(a.table, first + j / a.table.page_size);
    if (page < 0) page = 0;
    const uint8_t* src = a.cache + (static_cast<size_t>(page) * a.table.page_size + j % a.table.page_size) * kLatDk;
    const float sc = __ldg(a.scale + page);
    const uint4 x = *reinterpret_cast<const uint4*>(src + lane * 16);
    float v[16];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    for (int k = 0; k < 4; ++k) {
      const float4 f = e4m3x4_to_float(w[k]);
      v[4 * k] = f.x; v[4 * k + 1] = f.y; v[4 * k + 2] = f.z; v[4 * k + 3] = f.w;
    }
    const float4 rot = e4m3x4_to_float(*reinterpret_cast<const uint16_t*>(src + 512 + 2 * lane));
    float s = q[16] * rot.x + q[17] * rot.y;
    for (int k = 0; k < 16; ++k) s += q[k] * v[k];
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= sc * a.sm_scale;
    if (a.logit_cap > 0.0f) s = a.logit_cap * tanhf(s / a.logit_cap);
    s *= kLog2e;
    const float mn = fmaxf(m, s), alpha = exp2f(m - mn), p = exp2f(s - mn);
    l = l * alpha + p;
    for (int k = 0; k < 16; ++k) acc[k] = acc[k] * alpha + p * sc * v[k];
    m = mn;
  }
  const float inv = sees > 0 ? 1.0f / l : 0.0f;
  for (int k = 0; k < 16; ++k) a.o[row * kLatDv + lane * 16 + k] = __float2bfloat16(acc[k] * inv);
  if (a.lse && lane == 0) a.lse[row] = sees > 0 ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace fp8moe
