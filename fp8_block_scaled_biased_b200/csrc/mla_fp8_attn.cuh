// Multi-head latent attention over the 8-bit paged latent cache, for one query token per
// sequence (decode) and for several with a causal mask (extend).
//
//   s_j = sm_scale * <q, k_j> over 576 entries, soft-capped if asked;  o = softmax(s) V,
//   V the first 512 entries of the same rows.
//
// Both products run on the FP8 tensor cores straight from the cache's codes: nothing is
// dequantised. Tokens and value columns are the M of the MMAs, (query, head) columns are N:
//   S^T [128 tokens, N] = K [128, 576] Q^T        A = the tile as it lies (K-major)
//   O^T [512 values, N] += V^T [512, 128] P^T     A = the same shared memory, read M-major
// so 16 heads fill an MMA as well as 128 would. The bf16 and fp32 operands become sums of e4m3
// codes, each term its own N column, joined after the MMA in fp32:
//   q / s = hi + lo / 16, s a power of two per (query, head): hi is q / s rounded, and the
//     rest of an 8-bit significand is exactly a 4-bit one (until lo falls to subnormals,
//     2^-13 below the row's largest entry). N = 2 x columns.
//   p = hi + lo / 32 + lo2 / 1024: 12 bits, down to 2^-25 of the largest weight, so that a
//     long faint context beside one dominant token keeps its mass. N = 3 x columns.
// Products of codes are exact and the MMA sums in fp32. Scales of pages (one per token row,
// i.e. per TMEM lane) multiply the scores, and the weights before they are split.
//
// A CTA holds `HG` columns and walks 128-token tiles through two shared-memory stages:
//   warp 0      page table -> TMA (boxes of 8 to 128 rows that a page holds together; gather4
//               for other page sizes), and the tokens' scales
//   warp 1      the MMAs: scores of the next tile are issued ahead of this tile's P V if its
//               rows have landed, else after
//   warp 2      the work list (below)
//   warps 4..   one warpgroup per 16 columns, a token per thread: online softmax. The running
//               reference of a column only moves when a score passes it by more than one
//               (base 2), and then the accumulators in TMEM are rescaled.
//
// Work list: the tiles of all (sequence, column group) pairs in one row, cut into equal
// shares; a share may begin and end inside a pair. Pairs cut in parts leave unnormalised
// fp32 partials (two per CTA at most) that a second kernel joins in order. Sequences with
// several column groups give them to a gang of G neighbouring CTAs that walk the same tiles
// at the same time, so that the rows come from HBM once and from L2 G - 1 times.
#pragma once

#include "gemm_sm100.cuh"
#include "mla_fp8_cache.cuh"

namespace fp8moe {

constexpr int kLatDv = 512;
constexpr int kLatTile = 128;                              // tokens per tile
constexpr int kLatStages = 2;
constexpr int kLatChunk = kLatTile * 128;                  // 128 bytes of every row of a tile
constexpr int kLatStageBytes = kLatTile * kLatDk;          // four chunks and the 64 rotary bytes
constexpr int kLatMaxCtas = 148;                           // one per SM
constexpr float kLatHeadroom = 1.0f;                       // a weight may pass its reference by 2^1
constexpr float kLatPExp = 7.0f;                           // reference weight as a code: 2^7, at most 2^8 <= 448

struct LatAttnArgs {
  const __nv_bfloat16* q;        // [num_q, Hq, 576]
  const int32_t* qo_indptr;      // [B + 1], or null: one query token per sequence
  const float* scale;
  PageTable table;
  __nv_bfloat16* o;              // [num_q, Hq, 512]
  float* lse;                    // [num_q, Hq] or null
  float* part_o;                 // [2 * CTAs, HG, 512]
  float2* part_ml;               // [2 * CTAs, HG]: reference and sum
  int4* merge;                   // [CTAs]: first row, columns, parts, first part's slot (parts 0: nothing)
  int num_q, Hq, gang;
  int run;                       // rows per TMA box (8 .. 128), or 0: gather4
  float sm_scale, logit_cap;
};

// One share of one column group's tiles.
struct LatFragment {
  int first;                     // its sequence's first page-table entry
  int len;                       // tokens of the sequence that some column sees
  int tile0, tile1;
  int row0, cols;                // its first row of q viewed as [num_q * Hq, 576], and how many
  int col0, sees0;               // column c sees sees0 + (col0 + c) / Hq tokens
  int slot;                      // where its partial goes; -1: it is whole
  int valid;                     // 0: the end of the list
};

template <int HG>
struct LatSmem {
  static constexpr int kQRows = 2 * HG, kPRows = 3 * HG;
  static constexpr int kQBytes = kQRows * kLatDk;
  static constexpr int kPBytes = kPRows * kLatTile;
  static constexpr int kOffQ = kLatStages * kLatStageBytes;
  static constexpr int kOffP = kOffQ + kQBytes;
  static constexpr int kOffInfo = kOffP + 2 * kPBytes;
  // TMEM columns: two score buffers, four accumulators of 128 value columns
  static constexpr int kTmemS = 0, kTmemO = 2 * kQRows;
  static constexpr int kTmemCols = (kTmemO + 4 * kPRows <= 256) ? 256 : 512;
  static constexpr int kThreads = 128 + 128 * (HG / 16);
  struct Info {
    LatFragment frag[2];
    float scale[kLatStages][kLatTile];
    float red[HG / 16][4][16];
    float red2[HG / 16][4][16];
    uint64_t kv_full[kLatStages], kv_empty[kLatStages], s_full[2], s_empty[2], p_full[2], p_empty[2];
    uint64_t frag_full[2], frag_empty[2], q_full;
    long long scan[kThreads / 32];
    long long start_off;          // position of the first sequence of this CTA's share
    int start_b;
    uint32_t tmem;
    int abort;
  };
  static constexpr int kBytes = kOffInfo + static_cast<int>(sizeof(Info)) + 1024;   // + alignment
};

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ void tma_gather4(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int4 rows) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z),
      "r"(rows.w)
      : "memory");
}
// 32 lanes x N consecutive fp32 columns, waited for.
__device__ __forceinline__ void tmem_load_32(uint32_t taddr, float (&v)[32]) {
  tmem_ld_32x32b_x32(taddr, v);
  tmem_wait_ld();
  reg_fence_32(v);
}
__device__ __forceinline__ void tmem_load_16(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_store_16(uint32_t taddr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory descriptor: start, the two strides between core matrices, swizzle (0 none, 2: 128 B, 4: 64 B).
__device__ __forceinline__ uint64_t umma_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1u) << 46) |
         (static_cast<uint64_t>(layout) << 61);
}
// Barrier of one warpgroup (named barrier `id`) that ors a predicate.
__device__ __forceinline__ bool group_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(id)
      : "memory");
  return r != 0;
}
// Whether a phase has completed, without waiting for it (try_wait may suspend the thread).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp16 -> two e4m3 codes, and back.
__device__ __forceinline__ uint16_t half2_to_e4m3x2(__half2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
  return r;
}
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return *reinterpret_cast<const __half2*>(&r);
}

// ---------------------------------------------------------------- work list
struct LatShape {
  int first, len, qlo, n;        // page-table entry, tokens, first query row, query tokens
  int units, groups, tiles;      // column groups, gangs of them, tiles of each
};

// A sequence's share of the work list; one with no query or a bad table has none.
__device__ __forceinline__ LatShape lat_shape(const LatAttnArgs& a, int b, int HG) {
  LatShape s{};
  s.qlo = b;
  s.n = 1;
  if (a.qo_indptr) {
    const int lo = __ldg(a.qo_indptr + b), hi = __ldg(a.qo_indptr + b + 1);
    if (lo < 0 || hi < lo || hi > a.num_q) {
      raise_device_error(FP8MOE_DEVERR_PAGE);
      s.n = 0;
      return s;
    }
    s.qlo = lo;
    s.n = hi - lo;
  }
  if (!sequence_extent(a.table, b, s.first, s.len)) s.n = 0;
  if (s.n == 0) return s;
  const long long cols = static_cast<long long>(s.n) * a.Hq;
  s.units = static_cast<int>((cols + HG - 1) / HG);
  s.groups = (s.units + a.gang - 1) / a.gang;
  s.tiles = max(1, (s.len + kLatTile - 1) / kLatTile);     // an empty sequence still writes its rows
  return s;
}

// Warp 2, one lane: the fragments of positions [p0, p1) of the work list, through the ring.
template <int HG>
__device__ __forceinline__ bool lat_schedule(const LatAttnArgs& a, typename LatSmem<HG>::Info* s, long long total,
                                             int ngangs, int gang_id, int rank) {
  const long long p0 = total * gang_id / ngangs, p1 = total * (gang_id + 1) / ngangs;
  int b = s->start_b;
  long long off = s->start_off;
  LatShape sh{};
  if (p0 < p1) sh = lat_shape(a, b, HG);
  int slot = 0, merge_parts = 0, merge_slot = 0, merge_row = 0, merge_cols = 0;
  uint32_t phase = 0;
  auto push = [&](const LatFragment& f) {
    if (!mbar_wait_idle(&s->frag_empty[slot], phase ^ 1u, &s->abort)) return false;
    s->frag[slot] = f;
    mbar_arrive(&s->frag_full[slot]);
    if (++slot == 2) { slot = 0; phase ^= 1u; }
    return true;
  };
  for (long long p = p0; p < p1;) {
    while (p >= off + static_cast<long long>(sh.groups) * sh.tiles) {
      off += static_cast<long long>(sh.groups) * sh.tiles;
      sh = lat_shape(a, ++b, HG);
    }
    const int v = static_cast<int>((p - off) / sh.tiles);
    const long long base = off + static_cast<long long>(v) * sh.tiles;
    const int t0 = static_cast<int>(p - base);
    const int t1 = static_cast<int>(min(static_cast<long long>(sh.tiles), p1 - base));
    // early and late column groups in turn: what a causal mask takes from one share it takes from all
    const int g = (v & 1) ? sh.groups - 1 - v / 2 : v / 2;
    const int u = g * a.gang + rank;
    p = base + t1;
    if (u >= sh.units) continue;
    LatFragment f{};
    f.first = sh.first;
    f.col0 = u * HG % a.Hq;
    const long long c0 = static_cast<long long>(u) * HG, cols = static_cast<long long>(sh.n) * a.Hq;
    f.cols = static_cast<int>(min(static_cast<long long>(HG), cols - c0));
    f.row0 = static_cast<int>(static_cast<long long>(sh.qlo) * a.Hq + c0);
    f.sees0 = sh.len - sh.n + static_cast<int>(c0 / a.Hq) + 1;
    f.len = max(0, min(sh.len, f.sees0 + (f.col0 + f.cols - 1) / a.Hq));
    const int tiles = max(1, (f.len + kLatTile - 1) / kLatTile);
    f.tile0 = t0;
    f.tile1 = min(t1, tiles);
    if (f.tile0 >= f.tile1) continue;
    f.slot = -1;
    f.valid = 1;
    if (f.tile0 > 0 || f.tile1 < tiles) {
      f.slot = 2 * blockIdx.x + (base + t0 == p0 ? 0 : 1);
      if (f.tile0 == 0) {        // the first part: this CTA's entry for the joining kernel
        const long long last = base + tiles - 1;           // the gang that holds the last tile
        merge_parts = static_cast<int>(((last + 1) * ngangs + total - 1) / total - 1) - gang_id + 1;
        merge_slot = f.slot;
        merge_row = f.row0;
        merge_cols = f.cols;
      }
    }
    if (!push(f)) return false;
  }
  a.merge[blockIdx.x] = make_int4(merge_row, merge_cols, merge_parts, merge_slot);
  return push(LatFragment{});
}

// ---------------------------------------------------------------- softmax warpgroup
// Codes of columns 2i and 2i + 1 (two bytes) of the three terms of y in [0, 2^8].
__device__ __forceinline__ void split_weights(float y0, float y1, uint16_t& hi, uint16_t& lo, uint16_t& lo2) {
  hi = cvt_e4m3x2(y0, y1);
  const float2 h = __half22float2(e4m3x2_to_half2(hi));
  // the rest is within half a step of hi: exact in fp32, 11 bits of it in fp16 (times 32: at most 256)
  const __half2 r = __floats2half2_rn((y0 - h.x) * 32.0f, (y1 - h.y) * 32.0f);
  lo = half2_to_e4m3x2(r);
  lo2 = half2_to_e4m3x2(__hmul2(__hsub2(r, e4m3x2_to_half2(lo)), __float2half2_rn(32.0f)));
}

__device__ __forceinline__ int float_order(float x) {      // order of floats as order of ints
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float order_float(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

template <int HG>
__device__ __forceinline__ bool lat_softmax_role(const LatAttnArgs& a, typename LatSmem<HG>::Info* s, uint8_t* smem,
                                                 uint32_t tmem) {
  using SM = LatSmem<HG>;
  volatile int* abort_flag = &s->abort;
  const int tid = threadIdx.x & 127, group = (threadIdx.x >> 7) - 1;   // warpgroup of 16 columns
  const int warp = tid >> 5, lane = tid & 31;
  const int bar_id = 1 + group;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  const bool capped = a.logit_cap > 0.0f;
  int fslot = 0;
  uint32_t fphase = 0;
  int it = 0;                                              // tiles so far: buffers and phases follow it

  for (;;) {
    bool ok = mbar_wait(&s->frag_full[fslot], fphase, abort_flag);
    if (group_any(bar_id, !ok)) return false;
    const LatFragment f = s->frag[fslot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&s->frag_empty[fslot]);
    if (++fslot == 2) { fslot = 0; fphase ^= 1u; }
    if (!f.valid) return true;

    // ---- the queries: eight threads per column, 72 entries each. The earlier fragment's score
    // MMAs are done (its last s_full was waited for), so their operand may be overwritten.
    float qf;                                              // of column tid / 8
    {
      const int c = group * 16 + (tid >> 3), part = tid & 7;
      const bool live = c < f.cols;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (static_cast<size_t>(f.row0) + (live ? c : 0)) * kLatDk) + part;
      uint4 x[9];
#pragma unroll
      for (int j = 0; j < 9; ++j) x[j] = live ? __ldg(src + 8 * j) : make_uint4(0, 0, 0, 0);
      uint32_t mx = 0;
#pragma unroll
      for (int j = 0; j < 9; ++j)
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(finite_magnitudes(x[j].x), finite_magnitudes(x[j].y)),
                                   __vmaxu2(finite_magnitudes(x[j].z), finite_magnitudes(x[j].w))));
      mx = max(mx & 0xffffu, mx >> 16);
      for (int d = 1; d < 8; d <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const int ex = max(kScaleMinExp, static_cast<int>(mx >> 7) - 135 + ((mx & 0x7fu) > 96u ? 1 : 0));
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      qf = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
      uint8_t* qs = smem + SM::kOffQ;
      const int row_hi = group * 32 + (tid >> 3);          // the terms of 16 columns lie together
#pragma unroll
      for (int j = 0; j < 9; ++j) {
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 v = bf16x2_to_float(w[i]);
          v.x *= inv;
          v.y *= inv;
          if (isinf(v.x)) v.x = NAN;                       // no code is infinite
          if (isinf(v.y)) v.y = NAN;
          hi[i] = cvt_e4m3x2(v.x, v.y);
          const float2 h = __half22float2(e4m3x2_to_half2(hi[i]));
          lo[i] = cvt_e4m3x2((v.x - h.x) * 16.0f, (v.y - h.y) * 16.0f);
        }
        // 8-byte pieces of core matrices of 8 rows x 16 bytes
        const int k = (j * 8 + part) * 8;
        uint8_t* dst = qs + (k >> 4) * (SM::kQRows * 16) + (k & 8);
        *reinterpret_cast<uint2*>(dst + row_hi * 16) =
            make_uint2(hi[0] | (static_cast<uint32_t>(hi[1]) << 16), hi[2] | (static_cast<uint32_t>(hi[3]) << 16));
        *reinterpret_cast<uint2*>(dst + (row_hi + 16) * 16) =
            make_uint2(lo[0] | (static_cast<uint32_t>(lo[1]) << 16), lo[2] | (static_cast<uint32_t>(lo[3]) << 16));
      }
      if (part == 0) s->red[group][0][tid >> 3] = qf * (a.sm_scale * (capped ? 1.0f : kLog2e));
      fence_proxy_async_smem();
    }
    if (group_any(bar_id, false)) return false;
    if (tid == 0) mbar_arrive(&s->q_full);
    float fac[16], ref[16], sum[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      fac[c] = s->red[group][0][c];
      ref[c] = -INFINITY;
      sum[c] = 0.0f;
    }
    const int sees_min = f.sees0 + (f.col0 + group * 16) / a.Hq;       // of this group's first column
    const int col = f.col0 + group * 16;

    for (int tile = f.tile0; tile < f.tile1; ++tile, ++it) {
      const int buf = it & 1, stage = it % kLatStages;
      const uint32_t phase = (it >> 1) & 1, kv_phase = (it / kLatStages) & 1;
      ok = mbar_wait(&s->s_full[buf], phase, abort_flag) && mbar_wait(&s->kv_full[stage], kv_phase, abort_flag) &&
           mbar_wait(&s->p_empty[buf], phase ^ 1u, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      const float sc = s->scale[stage][tid];
      tc_fence_after();
      float v[32];
      tmem_load_32(lane_base + SM::kTmemS + buf * SM::kQRows + group * 32, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->s_empty[buf]);
      float t[16];
      bool bad = true;                                     // a NaN in this token's row makes every score NaN
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        t[c] = (v[c] + v[16 + c] * 0.0625f) * (fac[c] * sc);
        bad = bad && isnan(t[c]);
      }
      if (capped) {
#pragma unroll
        for (int c = 0; c < 16; ++c) t[c] = a.logit_cap * tanhf(t[c] / a.logit_cap) * kLog2e;
      }
      const int pos = tile * kLatTile + tid;
      if ((tile + 1) * kLatTile > sees_min || (tile + 1) * kLatTile > f.len) {
        int sees = sees_min, left = a.Hq - col % a.Hq;     // columns until the next query
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          if (pos >= min(sees, f.len)) t[c] = -INFINITY;
          if (--left == 0) { left = a.Hq; ++sees; }
        }
      }
      // the reference of a column bounds score + log2(page scale): the weights that meet the codes
      const float lg = sc > 0.0f ? log2f(sc) : -100.0f;
      bool over = false;
#pragma unroll
      for (int c = 0; c < 16; ++c) over = over || (t[c] + lg > ref[c] + kLatHeadroom);
      if (group_any(bar_id, over || !ok)) {
        if (group_any(bar_id, !ok)) return false;
        // new references: the largest over the tile, where that is larger
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float x = isnan(t[c]) ? -INFINITY : t[c] + lg;
          const int m = __reduce_max_sync(0xffffffffu, float_order(x));
          if (lane == 0) s->red2[group][warp][c] = order_float(m);
        }
        if (group_any(bar_id, false)) return false;
        float alpha[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float m = fmaxf(fmaxf(s->red2[group][0][c], s->red2[group][1][c]),
                                fmaxf(s->red2[group][2][c], s->red2[group][3][c]));
          const float next = fmaxf(ref[c], m);
          alpha[c] = next == -INFINITY ? 1.0f : exp2_fast(ref[c] - next);
          ref[c] = next;
          sum[c] *= alpha[c];
        }
        if (tile > f.tile0) {                              // what has been summed, in the new references
          ok = mbar_wait(&s->p_empty[buf ^ 1], ((it - 1) >> 1) & 1, abort_flag);
          if (group_any(bar_id, !ok)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int term = 0; term < 3; ++term) {
              const uint32_t at = lane_base + SM::kTmemO + m * SM::kPRows + group * 48 + term * 16;
              float w[16];
              tmem_load_16(at, w);
#pragma unroll
              for (int c = 0; c < 16; ++c) w[c] *= alpha[c];
              tmem_store_16(at, w);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        if (group_any(bar_id, false)) return false;        // red2 may be written again
      }
      // weights, their sum, and their codes: 16 bytes per term and token
      uint32_t code[3][4];
      const float gain = sc;
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const float r0 = ref[c] == -INFINITY ? 0.0f : ref[c], r1 = ref[c + 1] == -INFINITY ? 0.0f : ref[c + 1];
        const float p0 = exp2_fast(t[c] - r0 + kLatPExp), p1 = exp2_fast(t[c + 1] - r1 + kLatPExp);
        sum[c] += p0;
        sum[c + 1] += p1;
        uint16_t hi, lo, lo2;
        split_weights(p0 * gain, p1 * gain, hi, lo, lo2);
        const int w = c >> 2, sh = (c & 2) * 8;
        if (sh == 0) {
          code[0][w] = hi;
          code[1][w] = lo;
          code[2][w] = lo2;
        } else {
          code[0][w] |= static_cast<uint32_t>(hi) << 16;
          code[1][w] |= static_cast<uint32_t>(lo) << 16;
          code[2][w] |= static_cast<uint32_t>(lo2) << 16;
        }
      }
      uint8_t* pb = smem + SM::kOffP + buf * SM::kPBytes + group * 3 * (16 * kLatTile) + tid * 16;
#pragma unroll
      for (int term = 0; term < 3; ++term)
        *reinterpret_cast<uint4*>(pb + term * (16 * kLatTile)) =
            make_uint4(code[term][0], code[term][1], code[term][2], code[term][3]);
      if (bad) {
        // the row must not reach columns that give it no weight (0 x NaN): its values become 0, the
        // weights of the columns that do see it are NaN themselves
        uint8_t* row = smem + stage * kLatStageBytes + tid * 128;
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
          *reinterpret_cast<uint4*>(row + (i >> 3) * kLatChunk + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->p_full[buf]);
    }

    // ---- the fragment's result: the columns' sums over all threads, then the accumulators
    const int lastbuf = (it - 1) & 1;
    ok = mbar_wait(&s->p_empty[lastbuf], ((it - 1) >> 1) & 1, abort_flag);
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      float x = sum[c];
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      if (lane == 0) s->red2[group][warp][c] = x;
    }
    if (group_any(bar_id, !ok)) return false;
#pragma unroll
    for (int c = 0; c < 16; ++c)
      sum[c] = (s->red2[group][0][c] + s->red2[group][1][c]) + (s->red2[group][2][c] + s->red2[group][3][c]);
    tc_fence_after();
    const int live = min(16, f.cols - group * 16);
    const size_t row0 = static_cast<size_t>(f.row0) + group * 16;
    const size_t part0 = static_cast<size_t>(max(f.slot, 0)) * HG + group * 16;
#pragma unroll 1
    for (int m = 0; m < 4; ++m) {
      float acc[16], w[16];
      const uint32_t at = lane_base + SM::kTmemO + m * SM::kPRows + group * 48;
      tmem_load_16(at + 32, acc);
      tmem_load_16(at + 16, w);
#pragma unroll
      for (int c = 0; c < 16; ++c) acc[c] = w[c] + acc[c] * 0.03125f;
      tmem_load_16(at, w);
#pragma unroll
      for (int c = 0; c < 16; ++c) acc[c] = w[c] + acc[c] * 0.03125f;
      const int d = m * 128 + tid;
      if (f.slot < 0) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c < live)
            a.o[(row0 + c) * kLatDv + d] = __float2bfloat16(sum[c] == 0.0f ? 0.0f : acc[c] / sum[c]);
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c < live) a.part_o[(part0 + c) * kLatDv + d] = acc[c];
      }
    }
    tc_fence_before();
    if (tid < 16 && tid < live) {
      float m = 0.0f, l = 0.0f;
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (c == tid) { m = ref[c]; l = sum[c]; }
      if (f.slot >= 0) {
        a.part_ml[part0 + tid] = make_float2(m, l);
      } else if (a.lse) {
        a.lse[row0 + tid] = l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) - kLatPExp + log2f(l)) * kLn2;
      }
    }
  }
}

// ---------------------------------------------------------------- the kernel
template <int HG>
__global__ void __launch_bounds__(LatSmem<HG>::kThreads, 1)
mla_fp8_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rot,
               const __grid_constant__ LatAttnArgs a) {
  using SM = LatSmem<HG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  typename SM::Info* s = reinterpret_cast<typename SM::Info*>(smem + SM::kOffInfo);
  volatile int* abort_flag = &s->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kGroups = HG / 16;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kLatStages; ++i) {
      mbar_init(&s->kv_full[i], 1);
      mbar_init(&s->kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s->s_full[i], 1);
      mbar_init(&s->s_empty[i], 4 * kGroups);
      mbar_init(&s->p_full[i], 4 * kGroups);
      mbar_init(&s->p_empty[i], 1);
      mbar_init(&s->frag_full[i], 1);
      mbar_init(&s->frag_empty[i], 2 + 4 * kGroups);
    }
    mbar_init(&s->q_full, kGroups);
    s->abort = 0;
    s->start_b = 0;
    s->start_off = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_lat);
    prefetch_tensormap(&tm_rot);
  }
  if (warp == 1) {
    tmem_alloc(&s->tmem, SM::kTmemCols);
    tmem_relinquish();
  }
  // the work list's length, and the sequence that this CTA's share begins in: a run of
  // sequences per thread, then a scan over the threads
  const int per = (a.table.B + SM::kThreads - 1) / SM::kThreads;
  const int b0 = threadIdx.x * per, b1 = min(a.table.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const LatShape sh = lat_shape(a, b, HG);
    mine += static_cast<long long>(sh.groups) * sh.tiles;
  }
  long long incl = mine;
  for (int d = 1; d < 32; d <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += up;
  }
  if (lane == 31) s->scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < SM::kThreads / 32; ++w) {
    if (w < warp) before += s->scan[w];
    total += s->scan[w];
  }
  const int gang_id = blockIdx.x / a.gang, rank = blockIdx.x % a.gang;
  const int ngangs = static_cast<int>(min(static_cast<long long>(gridDim.x / a.gang), total));
  const bool works = gang_id < ngangs;
  if (works) {
    const long long p0 = total * gang_id / ngangs;
    if (p0 >= before && p0 < before + mine) {
      long long off = before;
      for (int b = b0; b < b1; ++b) {
        const LatShape sh = lat_shape(a, b, HG);
        const long long w = static_cast<long long>(sh.groups) * sh.tiles;
        if (p0 < off + w) {
          s->start_b = b;
          s->start_off = off;
          break;
        }
        off += w;
      }
    }
  }
  __syncthreads();
  const uint32_t tmem = s->tmem;
  bool ok = true;

  if (!works) {
    if (threadIdx.x == 0) a.merge[blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (warp >= 4) {
    ok = lat_softmax_role<HG>(a, s, smem, tmem);
  } else if (warp == 2) {
    if (lane == 0) ok = lat_schedule<HG>(a, s, total, ngangs, gang_id, rank);
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------ rows and scales
    int it = 0, fslot = 0;
    uint32_t fphase = 0;
    const int ps = a.table.page_size, run = a.run;
    for (;;) {
      ok = __all_sync(0xffffffffu, mbar_wait(&s->frag_full[fslot], fphase, abort_flag));
      if (!ok) break;
      const LatFragment f = s->frag[fslot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->frag_empty[fslot]);
      if (++fslot == 2) { fslot = 0; fphase ^= 1u; }
      if (!f.valid) break;
      for (int tile = f.tile0; tile < f.tile1; ++tile, ++it) {
        const int stage = it % kLatStages;
        const int tok = tile * kLatTile;
        // this lane's rows (a run of them, or four) and their scales, before the stage is free
        int4 rows = make_int4(0, 0, 0, 0);
        float4 sc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        bool live;
        if (run) {
          const int pos = tok + lane * run;
          live = lane < kLatTile / run && pos < f.len;
          float one = 0.0f;
          if (live) {
            const int page = table_page(a.table, f.first + pos / ps);
            live = page >= 0;
            if (live) {
              rows.x = page * ps + pos % ps;
              one = __ldg(a.scale + page);
            }
          }
          one = __shfl_sync(0xffffffffu, one, 4 * lane / run);
          sc = make_float4(one, one, one, one);
        } else {
          const int pos = tok + 4 * lane;
          live = pos < f.len;
          int* r = reinterpret_cast<int*>(&rows);
          float* c = reinterpret_cast<float*>(&sc);
          int fallback = -1;                               // a row past the end repeats one before it
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int p = min(pos + i, f.len - 1);
            if (live) {
              const int page = table_page(a.table, f.first + p / ps);
              if (page >= 0) {
                fallback = page * ps + p % ps;
                c[i] = __ldg(a.scale + page);
              }
              r[i] = fallback;
            }
          }
          if (live && fallback < 0) live = false;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (r[i] < 0) r[i] = max(fallback, 0);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&s->kv_empty[stage], ((it / kLatStages) & 1) ^ 1u, abort_flag));
        if (!ok) break;
        *reinterpret_cast<float4*>(&s->scale[stage][4 * lane]) = sc;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * (run ? run : 4) * kLatDk;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&s->kv_full[stage], bytes);
        __syncwarp();
        if (live) {
          uint8_t* dst = smem + stage * kLatStageBytes;
          const int at = lane * (run ? run : 4);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (run) tma_load_2d(dst + c * kLatChunk + at * 128, &tm_lat, &s->kv_full[stage], c * 128, rows.x);
            else tma_gather4(dst + c * kLatChunk + at * 128, &tm_lat, &s->kv_full[stage], c * 128, rows);
          }
          if (run) tma_load_2d(dst + 4 * kLatChunk + at * 64, &tm_rot, &s->kv_full[stage], 512, rows.x);
          else tma_gather4(dst + 4 * kLatChunk + at * 64, &tm_rot, &s->kv_full[stage], 512, rows);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    if (!ok) {
      // copies already in flight must land before the CTA's shared memory goes away
      const unsigned long long t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 10000000ull) {}
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (lane == 0) {
      constexpr uint32_t kIdescS = umma_idesc_e4m3_f32(128, SM::kQRows);
      constexpr uint32_t kIdescO = umma_idesc_e4m3_f32(128, SM::kPRows) | (1u << 15) | (1u << 16);   // A and B M/N-major
      const uint32_t base = smem_u32(smem);
      int it0 = 0, fslot = 0, fcount = 0;
      uint32_t fphase = 0;
      while (ok) {
        ok = mbar_wait(&s->frag_full[fslot], fphase, abort_flag);
        if (!ok) break;
        const int n = s->frag[fslot].tile1 - s->frag[fslot].tile0;
        const bool valid = s->frag[fslot].valid != 0;
        mbar_arrive(&s->frag_empty[fslot]);
        if (++fslot == 2) { fslot = 0; fphase ^= 1u; }
        if (!valid) break;
        ok = mbar_wait(&s->q_full, fcount & 1, abort_flag);
        ++fcount;
        if (!ok) break;
        int qk = 0, pv = 0;
        unsigned long long t0 = global_timer_ns();
        for (uint32_t spin = 0; pv < n; ++spin) {
          bool moved = false;
          if (qk < n && qk <= pv + 1) {
            const int i = it0 + qk, stage = i % kLatStages, buf = i & 1;
            if (mbar_test(&s->kv_full[stage], (i / kLatStages) & 1) &&
                mbar_test(&s->s_empty[buf], ((i >> 1) & 1) ^ 1u)) {
              tc_fence_after();
              const uint32_t kv = base + stage * kLatStageBytes, q = base + SM::kOffQ;
              const uint32_t d = tmem + SM::kTmemS + buf * SM::kQRows;
#pragma unroll 1
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  umma_f8(d, umma_desc(kv + c * kLatChunk + k * 32, 16, 1024, 2),
                          umma_desc(q + (c * 8 + k * 2) * (SM::kQRows * 16), SM::kQRows * 16, 128, 0), kIdescS,
                          (c | k) > 0 ? 1u : 0u);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                umma_f8(d, umma_desc(kv + 4 * kLatChunk + k * 32, 16, 512, 4),
                        umma_desc(q + (32 + k * 2) * (SM::kQRows * 16), SM::kQRows * 16, 128, 0), kIdescS, 1u);
              umma_commit(&s->s_full[buf]);
              ++qk;
              moved = true;
            }
          }
          if (pv < qk) {
            const int i = it0 + pv, stage = i % kLatStages, buf = i & 1;
            if (mbar_test(&s->p_full[buf], (i >> 1) & 1)) {
              tc_fence_after();
              const uint32_t kv = base + stage * kLatStageBytes, p = base + SM::kOffP + buf * SM::kPBytes;
#pragma unroll 1
              for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  umma_f8(tmem + SM::kTmemO + m * SM::kPRows,
                          umma_desc(kv + m * kLatChunk + k * 32 * 128, 1024, 1024, 2),
                          umma_desc(p + k * 32 * 16, 128, 16 * kLatTile, 0), kIdescO, (pv | k) > 0 ? 1u : 0u);
              umma_commit(&s->kv_empty[stage]);
              umma_commit(&s->p_empty[buf]);
              ++pv;
              moved = true;
            }
          }
          if (moved) {
            t0 = global_timer_ns();
          } else if ((spin & 63u) == 63u && (*abort_flag || global_timer_ns() - t0 > kWaitLimitNs)) {
            ok = false;
            break;
          }
        }
        it0 += n;
      }
    }
    __syncwarp();
  }
  if (!ok) {
    if (!*abort_flag) raise_device_error(FP8MOE_DEVERR_TIMEOUT);
    *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, SM::kTmemCols);
  }
}

// Joins the parts of the column groups that were cut: one block per (CTA that holds a first
// part, column), four value columns per thread; parts in order, so the same bits every time.
template <int HG>
__global__ void __launch_bounds__(128) mla_fp8_join_kernel(const LatAttnArgs a) {
  const int cta = blockIdx.x, c = blockIdx.y;
  const int4 job = a.merge[cta];
  if (job.z == 0 || c >= job.y) return;
  auto slot = [&](int i) { return static_cast<size_t>(i == 0 ? job.w : 2 * (cta + i * a.gang)) * HG + c; };
  float top = -INFINITY;
  for (int i = 0; i < job.z; ++i) {
    const float2 ml = a.part_ml[slot(i)];
    if (ml.y != 0.0f) top = fmaxf(top, ml.x);              // (a NaN sum has a reference too)
  }
  if (top == -INFINITY) top = 0.0f;
  float l = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = 0; i < job.z; ++i) {
    const size_t at = slot(i);
    const float2 ml = a.part_ml[at];
    if (ml.y == 0.0f) continue;
    const float w = exp2f((ml.x == -INFINITY ? 0.0f : ml.x) - top);
    const float4 x = reinterpret_cast<const float4*>(a.part_o + at * kLatDv)[threadIdx.x];
    l += w * ml.y;
    acc.x += w * x.x;
    acc.y += w * x.y;
    acc.z += w * x.z;
    acc.w += w * x.w;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t row = static_cast<size_t>(job.x) + c;
  __align__(8) __nv_bfloat162 y[2] = {__floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                                      __floats2bfloat162_rn(acc.z * inv, acc.w * inv)};
  reinterpret_cast<uint2*>(a.o + row * kLatDv)[threadIdx.x] = *reinterpret_cast<const uint2*>(y);
  if (a.lse && threadIdx.x == 0) a.lse[row] = l == 0.0f ? -INFINITY : (top - kLatPExp + log2f(l)) * 0.6931471805599453f;
}

}  // namespace fp8moe
