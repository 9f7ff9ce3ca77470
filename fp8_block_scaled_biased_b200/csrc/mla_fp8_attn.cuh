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
//   p = hi + lo / 32 + lo2 / 1024: off by 2^-12 of itself or 2^-22 of the largest weight, so that
//     a long faint context beside one dominant token keeps its mass. N = 3 x columns.
// Products of codes are exact and the MMA sums in fp32. Scales of pages (one per token row,
// i.e. per TMEM lane) multiply the scores, and the weights before they are split.
//
// A CTA holds `HG` columns and walks 128-token tiles through a ring of half tiles in shared memory:
//   warp 3      the work list (below) and the page table: the tiles' rows and scales, some tiles ahead
//   warp 0      TMA: boxes of 8 to 128 rows that a page holds together
//   warps 12-15 for smaller pages instead: 16-byte asynchronous copies
//   warps 1, 2  the MMAs: of the scores, and of P V
//   warps 4..   one warpgroup per 8 columns, a token per thread: online softmax. The running
//               reference of a column only moves when a weight would leave its code's range, and
//               then the accumulators in TMEM are rescaled.
//
// Work list: the tiles of all (sequence, column group) pairs in one row, cut into equal
// shares; a share may begin and end inside a pair. (Few and short sequences: one each.) Pairs
// cut in parts leave unnormalised fp32 partials (two per CTA at most) that a second kernel
// joins in order. Sequences with several column groups give them to a gang of G neighbouring
// CTAs that walk the same tiles at the same time, so that the rows come from HBM once and from
// L2 G - 1 times.
#pragma once

#include "gemm_sm100.cuh"
#include "mla_fp8_cache.cuh"

namespace fp8moe {

constexpr int kLatDv = 512;
constexpr int kLatTile = 128;                              // tokens per tile
constexpr int kLatChunk = kLatTile * 128;                  // 128 bytes of every row of a tile
constexpr int kLatHalf = 2 * kLatChunk;                    // two chunks: what is loaded and freed together
constexpr int kLatRot = kLatTile * 64;                     // the rotary bytes of a tile
constexpr int kLatMaxCtas = 148;                           // one per SM
// A weight's code runs up to 2^8 (of 448). Its column's reference stands at 2^2, so a score may pass the
// reference by 6 (base 2) before it has to move, which happens in about one tile of a hundred (of five,
// with 4). The smallest step of a code is 2^-19 (lo2's), so a weight is off by at most 2^-22 of the
// reference. Longer contexts, whose references settle early on, get a higher one, so that up to 2^18
// tokens together lose less than 2^-8 of it: half a step of the bf16 output.
__device__ __forceinline__ float lat_ref_exponent(int len) { return len <= (1 << 14) ? 2.0f : len <= (1 << 16) ? 4.0f : 6.0f; }
constexpr float kLatTopExp = 8.0f;
constexpr float kLatNoRef = 1e30f;                         // reference of a column that has none: any score passes it

struct LatAttnArgs {
  const __nv_bfloat16* q;        // [num_q, Hq, 576]
  const int32_t* qo_indptr;      // [B + 1], or null: one query token per sequence
  const uint8_t* cache;          // [num_pages * page_size, 576]
  const float* scale;
  PageTable table;
  __nv_bfloat16* o;              // [num_q, Hq, 512]
  float* lse;                    // [num_q, Hq] or null
  float* part_o;                 // [2 * CTAs, HG, 512]
  float2* part_ml;               // [2 * CTAs, HG]: reference and sum
  int4* merge;                   // [CTAs]: first row, columns, parts, first part's slot (parts 0: nothing)
  int num_q, Hq, gang_log;       // CTAs of a gang: 1, 2 or 4
  int run;                       // rows per TMA box: 8 to 128
  float sm_scale, logit_cap;
};

struct LatShape {
  int first, len, qlo, n;        // page-table entry, tokens, first query row, query tokens
  int units, groups, tiles;      // column groups, gangs of them, tiles of each
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
  // What shared memory holds: 2.5 tiles in halves (2 whole tiles cost 64 x 8192 tokens on 16 heads 7%),
  // the rotary bytes of two, the queries' terms, and the weights of two tiles, or of one beside 32
  // columns' queries.
  static constexpr int kHalves = 5, kRots = 2, kPBufs = HG == 16 ? 2 : 1;
  static constexpr int kAhead = HG == 16 ? 4 : 2;          // tiles whose page-table entries are fetched ahead
  static constexpr int kOffRot = kHalves * kLatHalf;
  static constexpr int kOffQ = kOffRot + kRots * kLatRot;
  static constexpr int kOffP = kOffQ + kQBytes;
  static constexpr int kOffInfo = kOffP + kPBufs * kPBytes;
  // TMEM columns: two score buffers, four accumulators of 128 value columns
  static constexpr int kTmemS = 0, kTmemO = 2 * kQRows;
  static constexpr int kTmemCols = (kTmemO + 4 * kPRows <= 256) ? 256 : 512;
  static constexpr int kGroups = HG / 8;                   // softmax warpgroups, 8 columns each
  struct Info {
    LatFragment frag[2];
    // per tile: the tokens' rows (or only those that begin a box), -1 for none; the tokens' scales
    union {
      int rows[kAhead][kLatTile];
      struct {                    // at the start only: the table warp reads it before it writes rows
        long long scan[24];
        int scan_most[24];
        long long start_off;      // position of the first sequence of this CTA's share,
        int start_b;              // the sequence, and its shape
        LatShape start;
      };
    };
    float scale[kAhead][kLatTile];
    int live[kAhead];             // rows to be loaded; -1: the end of the list
    uint64_t rows_full[kAhead], scale_full[kAhead], tab_empty[kAhead];
    float red[kGroups][4][8], qfac[kGroups][8];   // (of red, row 0 then holds reciprocals of the sums)
    uint64_t kv_full[kHalves], kv_empty[kHalves], rot_empty[kRots];
    uint64_t s_full[2], s_empty[2], p_full[kPBufs], p_empty[kPBufs];
    uint64_t frag_full[2], frag_empty[2], q_full;
    uint32_t tmem;
    int abort;
  };
  // 1 KB to align the start, where there is room for it: dynamic shared memory starts aligned here (and
  // the kernel checks)
  static constexpr int kLimit = 227 * 1024, kUsed = kOffInfo + static_cast<int>(sizeof(Info));
  static constexpr int kBytes = kUsed + 1024 <= kLimit ? kUsed + 1024 : kLimit;
  static_assert(kUsed <= kLimit, "shared memory of a CTA");
};

template <int HG, bool SMALL>
constexpr int kLatThreads = 128 + 128 * LatSmem<HG>::kGroups + (SMALL ? 128 : 0);

// Position of a half of a tile in the ring: its slot, and the parity of the slot's use.
struct LatHalf {
  int slot;
  uint32_t phase;
};
template <int N>
__device__ __forceinline__ LatHalf lat_half(int n) {
  return {n % N, static_cast<uint32_t>(n / N) & 1u};
}

// ---------------------------------------------------------------- PTX
// tma_load_2d on shared-memory addresses computed once.
__device__ __forceinline__ void tma_load_at(uint32_t smem_dst, uint64_t map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_dst),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void cp_async_16(uint32_t smem_dst, const void* gmem_src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(gmem_src) : "memory");
}
// 32 lanes x consecutive fp32 columns (in one or two runs): loads are waited for once, stores are not.
__device__ __forceinline__ void tmem_load_16(uint32_t at0, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(at0)
      : "memory");
}
__device__ __forceinline__ void tmem_load_16_8(uint32_t at0, uint32_t at1, float (&v)[24]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%24];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%25];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23])
      : "r"(at0), "r"(at1)
      : "memory");
}
__device__ __forceinline__ void tmem_store_16_8(uint32_t at0, uint32_t at1, const float (&v)[24]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%24], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n\t"
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%25], {%16,%17,%18,%19,%20,%21,%22,%23};"
      ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
        "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]),
        "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "r"(at0), "r"(at1)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory descriptor: start, the two strides between core matrices, swizzle (0 none, 2: 128 B, 4: 64 B).
__device__ __forceinline__ uint64_t umma_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1u) << 46) |
         (static_cast<uint64_t>(layout) << 61);
}
// Barriers of one warpgroup (named barrier `id`); the second ors a predicate.
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
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
// mbar_wait, with all but the first question out of line: the roles wait in some twenty places, and
// the kernel's code should stay small beside the instruction cache.
__device__ __noinline__ bool lat_wait_more(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_wait(bar, parity, abort);
}
__device__ __forceinline__ bool lat_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait(bar, parity) || lat_wait_more(bar, parity, abort);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Whether a phase has completed, without waiting for it (try_wait may suspend the thread).
__device__ __forceinline__ bool mbar_test_at(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- work list
// A sequence's share of the work list; one with no query or a bad table has none.
__device__ __noinline__ LatShape lat_shape(const LatAttnArgs& a, int b, int HG) {
  LatShape s{};
  int qlo = b, qhi = b + 1;
  if (a.qo_indptr) {
    qlo = a.qo_indptr[b];
    qhi = a.qo_indptr[b + 1];
  }
  const bool table = sequence_extent(a.table, b, s.first, s.len);
  if (qlo < 0 || qhi < qlo || qhi > a.num_q) {
    raise_device_error(FP8MOE_DEVERR_PAGE);
    return s;
  }
  if (!table || qhi == qlo) return s;
  s.qlo = qlo;
  s.n = qhi - qlo;
  // at most 2^22 queries of 128 heads: fits 32 bits
  s.units = (s.n * a.Hq + HG - 1) / HG;
  s.groups = (s.units + (1 << a.gang_log) - 1) >> a.gang_log;
  s.tiles = max(1, (s.len + kLatTile - 1) / kLatTile);     // an empty sequence still writes its rows
  return s;
}

__device__ __noinline__ long long lat_div_large(long long a, long long b) { return a / b; }
// Quotient of non-negative 64-bit numbers that mostly fit 32 bits.
__device__ __forceinline__ long long lat_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return lat_div_large(a, b);
}

// The fragments of positions [p, p1) of the work list, one at a time.
template <int HG>
struct LatSchedule {
  LatShape sh;                   // of sequence b, whose share of the list begins at off
  int b;
  long long off, p, p0, p1, total;
  int ngangs, gang_id, rank;
  int4 merge;                    // this CTA's entry for the joining kernel

  __device__ __forceinline__ LatFragment next(const LatAttnArgs& a) {
    LatFragment f{};
    while (p < p1) {
      while (p >= off + static_cast<long long>(sh.groups) * sh.tiles) {
        off += static_cast<long long>(sh.groups) * sh.tiles;
        sh = lat_shape(a, ++b, HG);
      }
      const int v = sh.groups == 1 ? 0 : static_cast<int>(lat_div(p - off, sh.tiles));
      const long long base = off + static_cast<long long>(v) * sh.tiles;
      const int t0 = static_cast<int>(p - base);
      const int t1 = static_cast<int>(min(static_cast<long long>(sh.tiles), p1 - base));
      const bool begins = p == p0;
      p = base + t1;
      // early and late column groups in turn: what a causal mask takes from one share it takes from all
      const int u = (((v & 1) ? sh.groups - 1 - v / 2 : v / 2) << a.gang_log) + rank;
      if (u >= sh.units) continue;
      const int c0 = u * HG, query = sh.n == 1 ? 0 : c0 / a.Hq;
      f.first = sh.first;
      f.col0 = c0 - query * a.Hq;
      f.cols = min(HG, sh.n * a.Hq - c0);
      f.row0 = sh.qlo * a.Hq + c0;
      f.sees0 = sh.len - sh.n + query + 1;
      f.len = max(0, min(sh.len, f.sees0 + (sh.n == 1 ? 0 : (f.col0 + f.cols - 1) / a.Hq)));
      const int tiles = max(1, (f.len + kLatTile - 1) / kLatTile);
      f.tile0 = t0;
      f.tile1 = min(t1, tiles);
      if (f.tile0 >= f.tile1) continue;
      f.slot = -1;
      f.valid = 1;
      if (f.tile0 > 0 || f.tile1 < tiles) {
        f.slot = 2 * blockIdx.x + (begins ? 0 : 1);
        if (f.tile0 == 0) {      // the first part; the last tile's gang says how many there are
          const int last_gang = static_cast<int>(lat_div((base + tiles) * ngangs + total - 1, total)) - 1;
          merge = make_int4(f.row0, f.cols, last_gang - gang_id + 1, f.slot);
        }
      }
      return f;
    }
    return LatFragment{};
  }
};

// ---------------------------------------------------------------- softmax warpgroup
// Four values as four codes per term; halves of words are handled as such, without 16-bit arithmetic.
// Weights in [0, 2^8]: rounded to the 11 bits of fp16, of which hi takes 4, lo 4 and lo2 the rest,
// exactly (down to lo2's subnormals): y = hi + lo / 32 + lo2 / 1024. The rest after a term is at most
// half its last step, so 32 times that fits the next.
__device__ __forceinline__ void split_weights(float y0, float y1, float y2, float y3, uint32_t& hi, uint32_t& lo,
                                              uint32_t& lo2) {
  asm("{\n\t.reg .b32 a, b, x, y, k;\n\t.reg .b16 p, q;\n\t"
      "mov.b32 k, 0x50005000;\n\t"                          // 32, 32
      "cvt.rn.f16x2.f32 a, %4, %3;\n\tcvt.rn.f16x2.f32 b, %6, %5;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, a;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, b;\n\tmov.b32 %0, {p, q};\n\t"
      "cvt.rn.f16x2.e4m3x2 x, p;\n\tcvt.rn.f16x2.e4m3x2 y, q;\n\t"
      "sub.rn.f16x2 a, a, x;\n\tsub.rn.f16x2 b, b, y;\n\tmul.rn.f16x2 a, a, k;\n\tmul.rn.f16x2 b, b, k;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, a;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, b;\n\tmov.b32 %1, {p, q};\n\t"
      "cvt.rn.f16x2.e4m3x2 x, p;\n\tcvt.rn.f16x2.e4m3x2 y, q;\n\t"
      "sub.rn.f16x2 a, a, x;\n\tsub.rn.f16x2 b, b, y;\n\tmul.rn.f16x2 a, a, k;\n\tmul.rn.f16x2 b, b, k;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, a;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, b;\n\tmov.b32 %2, {p, q};\n\t}"
      : "=r"(hi), "=r"(lo), "=r"(lo2)
      : "f"(y0), "f"(y1), "f"(y2), "f"(y3));
}
// Query entries of at most 448 in magnitude: x = hi + lo / 16.
__device__ __forceinline__ void split_query(float x0, float x1, float x2, float x3, uint32_t& hi, uint32_t& lo) {
  asm("{\n\t.reg .b32 a, b, x, y, k;\n\t.reg .b16 p, q;\n\t"
      "mov.b32 k, 0x4c004c00;\n\t"                          // 16, 16
      "cvt.rn.f16x2.f32 a, %3, %2;\n\tcvt.rn.f16x2.f32 b, %5, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, a;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, b;\n\tmov.b32 %0, {p, q};\n\t"
      "cvt.rn.f16x2.e4m3x2 x, p;\n\tcvt.rn.f16x2.e4m3x2 y, q;\n\t"
      "sub.rn.f16x2 a, a, x;\n\tsub.rn.f16x2 b, b, y;\n\tmul.rn.f16x2 a, a, k;\n\tmul.rn.f16x2 b, b, k;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, a;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, b;\n\tmov.b32 %1, {p, q};\n\t}"
      : "=r"(hi), "=r"(lo)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
}

__device__ __forceinline__ int float_order(float x) {      // order of floats as order of ints
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float order_float(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

// One of a thread's columns chosen by a runtime index, without indexing registers.
__device__ __forceinline__ float pick8(const float (&v)[8], int i) {
  float x = v[0];
#pragma unroll
  for (int c = 1; c < 8; ++c) x = i == c ? v[c] : x;
  return x;
}

// A thread's share of its warpgroup's 8 query columns: 16 threads per column, 9 pieces of 4 entries
// each. Loaded while the fragment before is still being worked on.
template <int HG>
struct LatQueries {
  uint2 x[9];

  __device__ __forceinline__ void load(const LatAttnArgs& a, const LatFragment& f, int group, int tid) {
    const int c = group * 8 + (tid >> 4);
    // a column without a query repeats the fragment's first one: its result is not written
    const uint2* src =
        reinterpret_cast<const uint2*>(a.q + (static_cast<size_t>(f.row0) + (c < f.cols ? c : 0)) * kLatDk) + (tid & 15);
#pragma unroll
    for (int j = 0; j < 9; ++j) x[j] = src[j * 16];
  }

  // Splits the entries into their two terms and stores them as the score MMAs' B operand: core
  // matrices of 8 rows x 16 bytes, this group's rows being its 8 high terms, then its 8 low ones.
  // Returns the scale of column tid / 16. A row with an entry that is not finite gets codes of 0 and the
  // scale NaN, which makes all its scores NaN: a NaN before the scale is a cached token's.
  __device__ __forceinline__ float store(uint8_t* qs, int group, int tid) const {
    constexpr int kLead = LatSmem<HG>::kQRows * 16;        // from 16 entries to the next
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < 9; ++j) mx = __vmaxu2(mx, __vmaxu2(x[j].x & 0x7fff7fffu, x[j].y & 0x7fff7fffu));
    mx = max(mx & 0xffffu, mx >> 16);
    for (int d = 1; d < 16; d <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const int ex = max(kScaleMinExp, static_cast<int>(mx >> 7) - 135 + ((mx & 0x7fu) > 96u ? 1 : 0));
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
    uint8_t* dst = qs + ((tid & 15) >> 2) * kLead + (tid & 3) * 4 + (group * 16 + (tid >> 4)) * 16;
#pragma unroll
    for (int j = 0; j < 9; ++j, dst += 4 * kLead) {        // 64 entries on
      const float2 v0 = bf16x2_to_float(x[j].x), v1 = bf16x2_to_float(x[j].y);
      uint32_t hi, lo;                                     // (x / scale is exact in fp16 above 2^-16)
      split_query(v0.x * inv, v0.y * inv, v1.x * inv, v1.y * inv, hi, lo);
      if (mx >= 0x7f80u) hi = lo = 0u;
      *reinterpret_cast<uint32_t*>(dst) = hi;
      *reinterpret_cast<uint32_t*>(dst + 128) = lo;
    }
    return mx >= 0x7f80u ? NAN : __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
  }
};

template <int HG>
__device__ __forceinline__ bool lat_softmax_role(const LatAttnArgs& a, typename LatSmem<HG>::Info* s, uint8_t* smem,
                                                 uint32_t tmem) {
  using SM = LatSmem<HG>;
  volatile int* abort_flag = &s->abort;
  const int tid = threadIdx.x & 127, group = (threadIdx.x >> 7) - 1;   // warpgroup of 8 columns
  const int warp = tid >> 5, lane = tid & 31;
  const int bar_id = 1 + group;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  // The terms of two groups' weights share 48 N columns: hi and lo of the first, both lo2, hi and lo
  // of the second; 16 bytes of a token's weights are one block of 16 N columns.
  const int block = 3 * (group >> 1) + 2 * (group & 1), block2 = 3 * (group >> 1) + 1, half8 = 8 * (group & 1);
  const uint32_t acc1 = lane_base + SM::kTmemO + 16 * block, acc2 = lane_base + SM::kTmemO + 16 * block2 + half8;
  const float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  const bool capped = a.logit_cap > 0.0f;
  // cap tanh(x), x = t / cap, to 2^-19 of itself however small x is. Below 1/2 it is t times a polynomial in x^2
  // that interpolates tanh(x) / x (2^-23), which also takes caps whose reciprocal or product with log2(e) leaves
  // fp32's normal range; above, cap (1 - 2 / (1 + e^2x)), which cancels where x is small (a few 2^-24 of the
  // cap). Most warps need the first alone (500-query chunks capped at 50: 171 us; 173 with the second alone, 194
  // with tanhf).
  const float cap2 = fminf(a.logit_cap * kLog2e, 3.4e38f), cap_in = fminf(1.0f / a.logit_cap, 3.4e38f);
  int fslot = 0;
  uint32_t fphase = 0;
  int it = 0;                                              // tiles so far: buffers and phases follow it
  LatFragment f;
  bool ok;
  // The next fragment, its queries split and handed to the score MMAs. The MMAs of the fragment before
  // are done with theirs (its last s_full was waited for), and its accumulators are not concerned.
  auto next_fragment = [&](LatFragment& to) {
    ok = lat_wait(&s->frag_full[fslot], fphase, abort_flag);
    if (group_any(bar_id, !ok)) return false;
    to = s->frag[fslot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&s->frag_empty[fslot]);
    if (++fslot == 2) { fslot = 0; fphase ^= 1u; }
    if (!to.valid) return true;
    LatQueries<HG> queries;
    queries.load(a, to, group, tid);
    const float qscale = queries.store(smem + SM::kOffQ, group, tid);
    if ((tid & 15) == 0) s->qfac[group][tid >> 4] = qscale * (a.sm_scale * (capped ? 1.0f : kLog2e));
    fence_proxy_async_smem();
    group_sync(bar_id);
    if (tid == 0) mbar_arrive(&s->q_full);
    return true;
  };
  float nref[8], sum[8];         // of each column: code exponent of the reference minus the reference; sum of weights
  f.valid = 0;
  for (;;) {
    // the next fragment's queries first, so that its scores are on their way while this one's result (the
    // columns' sums over all threads, the accumulators) is written
    LatFragment next;
    if (!next_fragment(next)) return false;
    if (f.valid) {
      ok = lat_wait(&s->p_empty[(it - 1) % SM::kPBufs], ((it - 1) / SM::kPBufs) & 1, abort_flag);
      // lane bits 4 .. 2 choose a half of the columns each: four lanes end with parts of one column's sum
#pragma unroll
      for (int h = 4; h; h >>= 1) {
        const bool upper = (lane & (4 * h)) != 0;
#pragma unroll
        for (int c = 0; c < h; ++c) {
          const float keep = upper ? sum[c + h] : sum[c], give = upper ? sum[c] : sum[c + h];
          sum[c] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * h);
        }
      }
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 2);
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 1);
      if ((lane & 3) == 0) s->red[group][warp][lane >> 2] = sum[0];
      if (group_any(bar_id, !ok)) return false;
      tc_fence_after();
      const int live = min(8, f.cols - group * 8);
      const size_t row0 = static_cast<size_t>(f.row0) + group * 8;
      const size_t part0 = static_cast<size_t>(max(f.slot, 0)) * HG + group * 8;
      if (tid < 8) {
        const float l = (s->red[group][0][tid] + s->red[group][1][tid]) + (s->red[group][2][tid] + s->red[group][3][tid]);
        const float m = pick8(nref, tid);                    // l sums 2^(score + m)
        if (tid < live) {
          if (f.slot >= 0) a.part_ml[part0 + tid] = make_float2(m, l);
          else if (a.lse) a.lse[row0 + tid] = l == 0.0f ? -INFINITY : (log2f(l) - m) * kLn2;
        }
        s->red[group][0][tid] = l == 0.0f ? 0.0f : 1.0f / l;
      }
      group_sync(bar_id);
      if (f.slot < 0) {
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[c] = s->red[group][0][c];
        // neighbouring lanes share the work: the even one stores both values of columns 0 .. 3, the odd one
        // those of 4 .. 7 (half as many, twice as wide stores)
        const bool odd = lane & 1;
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + (row0 + (odd ? 4 : 0)) * kLatDv) + (tid >> 1);
        const int mine = live - (odd ? 4 : 0);
#pragma unroll 1
        for (int m = 0; m < 4; ++m, dst += 64) {
          float x[24];
          tmem_load_16_8(acc1 + m * SM::kPRows, acc2 + m * SM::kPRows, x);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float y = fmaf(fmaf(x[16 + c], 0.03125f, x[8 + c]), 0.03125f, x[c]) * sum[c];
            x[c] = sum[c] == 0.0f ? 0.0f : y;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? x[c] : x[4 + c], 1);
            const __nv_bfloat162 y = odd ? __floats2bfloat162_rn(other, x[4 + c]) : __floats2bfloat162_rn(x[c], other);
            if (c < mine) dst[c * (kLatDv / 2)] = *reinterpret_cast<const uint32_t*>(&y);
          }
        }
      } else {                                               // a part, as it stands
        float* dst = a.part_o + part0 * kLatDv + tid;
#pragma unroll 1
        for (int m = 0; m < 4; ++m, dst += 128) {
          float x[24];
          tmem_load_16_8(acc1 + m * SM::kPRows, acc2 + m * SM::kPRows, x);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < live) dst[c * kLatDv] = fmaf(fmaf(x[16 + c], 0.03125f, x[8 + c]), 0.03125f, x[c]);
        }
      }
      tc_fence_before();
      group_sync(bar_id);                                    // red, inv and TMEM are read before what comes next
    }
    if (!next.valid) return true;
    f = next;
    float fac[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      fac[c] = s->qfac[group][c];
      nref[c] = kLatNoRef;
      sum[c] = 0.0f;
    }
    const float ref_exp = lat_ref_exponent(f.len);
    const int query = a.Hq >= f.col0 + HG ? 0 : (f.col0 + group * 8) / a.Hq;
    const int sees_min = f.sees0 + query;                  // of this group's first column
    const int next_query = (query + 1) * a.Hq - (f.col0 + group * 8);  // columns until the next query

    for (int tile = f.tile0; tile < f.tile1; ++tile, ++it) {
      const int buf = it & 1, pbuf = it % SM::kPBufs;
      const uint32_t phase = (it >> 1) & 1;
      const int ahead = it % SM::kAhead;
      ok = lat_wait(&s->scale_full[ahead], (it / SM::kAhead) & 1, abort_flag);
      const float sc = s->scale[ahead][tid];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->tab_empty[ahead]);
      // the reference of a column bounds score + log2(page scale): the weights that meet the codes
      // (below 2^-90 they are counted as of that scale, so that a sum of weights cannot leave fp32)
      const float bound = kLatTopExp - fmaxf(__log2f(sc), -90.0f);
      float2 fs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) fs[i] = __fmul2_rn(make_float2(fac[2 * i], fac[2 * i + 1]), make_float2(sc, sc));
      if (SM::kPBufs == 2) ok = lat_wait(&s->p_empty[pbuf], ((it / SM::kPBufs) & 1) ^ 1u, abort_flag) && ok;
      ok = lat_wait(&s->s_full[buf], phase, abort_flag) && ok;
      __syncwarp();
      tc_fence_after();
      float t[8];
      bool bad;                                            // a NaN in this token's row (queries have none)
      {
        float v[16];
        tmem_load_16(lane_base + SM::kTmemS + buf * SM::kQRows + group * 16, v);
        tc_fence_before();
        bad = isnan(v[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = __fmul2_rn(__ffma2_rn(make_float2(v[8 + 2 * i], v[9 + 2 * i]), make_float2(0.0625f, 0.0625f),
                                                 make_float2(v[2 * i], v[2 * i + 1])),
                                      fs[i]);
          t[2 * i] = x.x;
          t[2 * i + 1] = x.y;
        }
      }
      if (capped) {
        float x[8], far = 0.0f;
        auto twice = [](float v) { return make_float2(v, v); };
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          const float2 u = __fmul2_rn(make_float2(t[c], t[c + 1]), twice(cap_in)), y = __fmul2_rn(u, u);
          float2 r = __ffma2_rn(y, twice(0.0179887526f), twice(-0.0533871129f));
          r = __ffma2_rn(y, r, twice(0.13330476f));
          r = __ffma2_rn(y, r, twice(-0.333333105f));
          r = __ffma2_rn(y, r, twice(1.0f));
          r = __fmul2_rn(r, __fmul2_rn(make_float2(t[c], t[c + 1]), twice(kLog2e)));
          x[c] = u.x;
          x[c + 1] = u.y;
          t[c] = r.x;
          t[c + 1] = r.y;
          far = fmaxf(far, fmaxf(fabsf(u.x), fabsf(u.y)));
        }
        if (__any_sync(0xffffffffu, far >= 0.5f)) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (fabsf(x[c]) >= 0.5f)
              t[c] = cap2 * fmaf(-2.0f, __fdividef(1.0f, 1.0f + exp2_fast(x[c] * (2.0f * kLog2e))), 1.0f);
        }
      }
      const int pos = tile * kLatTile + tid;
      if ((tile + 1) * kLatTile > min(sees_min, f.len)) {
        int sees = sees_min, left = next_query;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (pos >= min(sees, f.len)) t[c] = -INFINITY;
          if (--left == 0) { left = a.Hq; ++sees; }
        }
      }
      // The weights are computed before the group has agreed, in a barrier, that no score passes its
      // bound; if one does, the references move and they are computed again. A fragment's first tile has
      // no references yet: it takes them first. (fmaxf passes over NaN.)
      bool moves = tile == f.tile0;
      float w[8], top = -INFINITY;
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        const float2 x = __fadd2_rn(make_float2(t[c], t[c + 1]), make_float2(nref[c], nref[c + 1]));
        w[c] = x.x;
        w[c + 1] = x.y;
        top = fmaxf(top, fmaxf(x.x, x.y));
      }
      uint32_t hi[2], lo[2], lo2[2];
      for (;;) {
        if (moves) {
          // new references: the largest over the tile, where that is larger
          const float lg = kLatTopExp - bound;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float x = isnan(t[c]) ? -INFINITY : t[c] + lg;
            const int m = __reduce_max_sync(0xffffffffu, float_order(x));
            if (lane == 0) s->red[group][warp][c] = order_float(m);
          }
          if (tile == f.tile0) {
            if (lane == 0) mbar_arrive(&s->s_empty[buf]);
            if (SM::kPBufs == 1) ok = lat_wait(&s->p_empty[pbuf], ((it / SM::kPBufs) & 1) ^ 1u, abort_flag) && ok;
          } else {
            ok = lat_wait(&s->p_empty[(it - 1) % SM::kPBufs], ((it - 1) / SM::kPBufs) & 1, abort_flag) && ok;
          }
          if (group_any(bar_id, !ok)) return false;
          float alpha[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float m = fmaxf(fmaxf(s->red[group][0][c], s->red[group][1][c]),
                                  fmaxf(s->red[group][2][c], s->red[group][3][c]));
            const float next = fminf(nref[c], ref_exp - m);            // m = -inf: as it was
            alpha[c] = exp2_fast(next - nref[c]);
            nref[c] = next;
            sum[c] *= alpha[c];
            w[c] = t[c] + next;
          }
          group_sync(bar_id);                              // red may be written again
          if (tile > f.tile0) {                            // what has been summed, in the new references
            tc_fence_after();
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              float x[24];
              tmem_load_16_8(acc1 + m * SM::kPRows, acc2 + m * SM::kPRows, x);
#pragma unroll
              for (int i = 0; i < 24; ++i) x[i] *= alpha[i & 7];
              tmem_store_16_8(acc1 + m * SM::kPRows, acc2 + m * SM::kPRows, x);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = exp2_fast(w[c]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 y0 = __fmul2_rn(make_float2(w[4 * i], w[4 * i + 1]), make_float2(sc, sc));
          const float2 y1 = __fmul2_rn(make_float2(w[4 * i + 2], w[4 * i + 3]), make_float2(sc, sc));
          split_weights(y0.x, y0.y, y1.x, y1.y, hi[i], lo[i], lo2[i]);
        }
        if (moves) break;
        if (lane == 0) mbar_arrive(&s->s_empty[buf]);
        // the P V that read this buffer before is done
        if (SM::kPBufs == 1) ok = lat_wait(&s->p_empty[pbuf], ((it / SM::kPBufs) & 1) ^ 1u, abort_flag) && ok;
        if (!group_any(bar_id, top > bound || !ok)) break;
        if (group_any(bar_id, !ok)) return false;
        moves = true;
      }
      uint8_t* pb = smem + SM::kOffP + pbuf * SM::kPBytes + tid * 16;
      *reinterpret_cast<uint4*>(pb + block * (16 * kLatTile)) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
      *reinterpret_cast<uint2*>(pb + block2 * (16 * kLatTile) + half8) = make_uint2(lo2[0], lo2[1]);
      if (bad) {
        // the row must not reach columns that give it no weight (0 x NaN): its values become 0, the
        // weights of the columns that do see it are NaN themselves
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
          *reinterpret_cast<uint4*>(smem + lat_half<SM::kHalves>(2 * it + (i >> 4)).slot * kLatHalf +
                                    ((i >> 3) & 1) * kLatChunk + tid * 128 + ((i ^ tid) & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->p_full[pbuf]);
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        const float2 x = __fadd2_rn(make_float2(sum[c], sum[c + 1]), make_float2(w[c], w[c + 1]));
        sum[c] = x.x;
        sum[c + 1] = x.y;
      }
    }

  }
}

// ---------------------------------------------------------------- MMA warps
// Scores and P V are issued by a warp each, so that one's waits pass while the other's MMAs run: with
// both in one warp a tile of 32 columns took 3170 cycles, of which its MMAs 1770 and what lay between
// them 670 (chunks of 500 queries on 16 heads: 182 us instead of 162). All lanes run the loops and one
// elected lane issues, so that descriptors stay in uniform registers: 44 and 48 cycles per MMA (16
// columns), 70 from a divergent branch.
template <int HG>
__device__ __forceinline__ bool lat_score_role(typename LatSmem<HG>::Info* s, uint8_t* smem, uint32_t tmem_any) {
  using SM = LatSmem<HG>;
  volatile int* abort_flag = &s->abort;
  constexpr uint32_t kIdesc = umma_idesc_e4m3_f32(128, SM::kQRows);
  const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
  const uint64_t desc_k = umma_desc(base, 16, 1024, 2);                            // rows of 128 bytes, K-major
  const uint64_t desc_rot = umma_desc(base + SM::kOffRot, 16, 512, 4);             // rows of 64 bytes
  const uint64_t desc_q = umma_desc(base + SM::kOffQ, SM::kQRows * 16, 128, 0);
  const bool leader = elect_one();
  static_assert(SM::kRots == 2, "rotary bytes lie in the place of the score buffer's number");
  int slot = 0, buf = 0, fslot = 0;                        // places of the next half and its scores
  uint32_t phase = 0, buf_phase = 1, fphase = 0, q_phase = 0;
  for (;;) {
    if (!__all_sync(0xffffffffu, lat_wait(&s->frag_full[fslot], fphase, abort_flag))) return false;
    const int n = __shfl_sync(0xffffffffu, s->frag[fslot].valid ? s->frag[fslot].tile1 - s->frag[fslot].tile0 : 0, 0);
    if (leader) mbar_arrive(&s->frag_empty[fslot]);
    if (++fslot == 2) { fslot = 0; fphase ^= 1u; }
    if (n == 0) return true;
    if (!__all_sync(0xffffffffu, lat_wait(&s->q_full, q_phase, abort_flag))) return false;
    q_phase ^= 1u;
    for (int t = 0; t < n; ++t) {
      const uint32_t d = tmem + SM::kTmemS + buf * SM::kQRows;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        bool ok = lat_wait(&s->kv_full[slot], phase, abort_flag);
        if (half == 0) ok = ok && lat_wait(&s->s_empty[buf], buf_phase, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc_fence_after();
        if (leader) {
          if (half == 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              umma_f8(d, desc_rot + buf * (kLatRot >> 4) + k * 2, desc_q + (32 + k * 2) * SM::kQRows, kIdesc, k > 0 ? 1u : 0u);
            umma_commit(&s->rot_empty[buf]);
          }
          const uint64_t rows = desc_k + slot * (kLatHalf >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_f8(d, rows + (k >> 2) * (kLatChunk >> 4) + (k & 3) * 2, desc_q + (half * 16 + k * 2) * SM::kQRows, kIdesc, 1u);
          if (half == 1) umma_commit(&s->s_full[buf]);
        }
        __syncwarp();
        if (++slot == SM::kHalves) { slot = 0; phase ^= 1u; }
      }
      buf ^= 1;
      if (buf == 0) buf_phase ^= 1u;
    }
  }
}

template <int HG>
__device__ __forceinline__ bool lat_value_role(typename LatSmem<HG>::Info* s, uint8_t* smem, uint32_t tmem_any) {
  using SM = LatSmem<HG>;
  volatile int* abort_flag = &s->abort;
  constexpr uint32_t kIdesc = umma_idesc_e4m3_f32(128, SM::kPRows) | (1u << 15) | (1u << 16);   // A and B M/N-major
  const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
  const uint64_t desc_v = umma_desc(base, 1024, 1024, 2);                          // the scores' rows, M-major
  const uint64_t desc_p = umma_desc(base + SM::kOffP, 128, 16 * kLatTile, 0);
  const bool leader = elect_one();
  int slot = 0, pbuf = 0, fslot = 0;
  uint32_t phase = 0, fphase = 0;
  for (;;) {
    if (!__all_sync(0xffffffffu, lat_wait(&s->frag_full[fslot], fphase, abort_flag))) return false;
    const int n = __shfl_sync(0xffffffffu, s->frag[fslot].valid ? s->frag[fslot].tile1 - s->frag[fslot].tile0 : 0, 0);
    if (leader) mbar_arrive(&s->frag_empty[fslot]);
    if (++fslot == 2) { fslot = 0; fphase ^= 1u; }
    if (n == 0) return true;
    for (int t = 0; t < n; ++t) {
      if (!__all_sync(0xffffffffu, lat_wait(&s->p_full[pbuf], phase, abort_flag))) return false;
      tc_fence_after();
      if (leader) {
        const uint64_t p = desc_p + pbuf * (SM::kPBytes >> 4);
        const uint32_t more = t > 0 ? 1u : 0u;
        int half = slot;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f8(tmem + SM::kTmemO + m * SM::kPRows, desc_v + half * (kLatHalf >> 4) + (m & 1) * (kLatChunk >> 4) + k * 256,
                    p + k * 32, kIdesc, k > 0 ? 1u : more);
          if (m & 1) {
            umma_commit(&s->kv_empty[half]);
            half = half == SM::kHalves - 1 ? 0 : half + 1;
          }
        }
        umma_commit(&s->p_empty[pbuf]);
      }
      __syncwarp();
      slot = slot >= SM::kHalves - 2 ? slot + 2 - SM::kHalves : slot + 2;
      if (++pbuf == SM::kPBufs) { pbuf = 0; phase ^= 1u; }
    }
  }
}

// ---------------------------------------------------------------- page table and row loads
// Warp 3: the fragments, for all roles, and the rows and scales of their tiles, some tiles ahead of
// the loads. A lane looks up a box of rows (SMALL: its four tokens) and hands over four tokens' scales;
// the rows go first, the loads do not need the scales.
template <int HG, bool SMALL>
__device__ __forceinline__ bool lat_table_role(const LatAttnArgs& a, typename LatSmem<HG>::Info* s,
                                               LatSchedule<HG>& schedule) {
  using SM = LatSmem<HG>;
  volatile int* abort_flag = &s->abort;
  const int lane = threadIdx.x & 31;
  const int ps = a.table.page_size, run = a.run;
  int slot = 0, fslot = 0;
  uint32_t phase = 0, fphase = 0;
  for (;;) {
    const LatFragment f = schedule.next(a);                // (every lane computes it)
    if (!__all_sync(0xffffffffu, lat_wait(&s->frag_empty[fslot], fphase ^ 1u, abort_flag))) return false;
    if (lane == 0) {
      s->frag[fslot] = f;
      mbar_arrive(&s->frag_full[fslot]);
      if (!f.valid) a.merge[blockIdx.x] = schedule.merge;
    }
    if (++fslot == 2) { fslot = 0; fphase ^= 1u; }
    const int tile1 = f.valid ? f.tile1 : f.tile0 + 1;     // the end takes an entry too
    for (int tile = f.tile0; tile < tile1; ++tile) {
      const int pos = tile * kLatTile + lane * (SMALL ? 4 : run);
      int page[SMALL ? 4 : 1], rows[SMALL ? 4 : 1];
      int at = pos / ps, off = pos - at * ps;
#pragma unroll
      for (int i = 0; i < (SMALL ? 4 : 1); ++i) {
        page[i] = -1;
        if (pos + i < f.len && (SMALL || lane < kLatTile / run)) page[i] = table_page(a.table, f.first + at);
        rows[i] = page[i] < 0 ? -1 : page[i] * ps + off;
        if (++off == ps) { off = 0; ++at; }
      }
      if (!__all_sync(0xffffffffu, lat_wait(&s->tab_empty[slot], phase ^ 1u, abort_flag))) return false;
      if constexpr (SMALL) {
        *reinterpret_cast<int4*>(&s->rows[slot][4 * lane]) = make_int4(rows[0], rows[1], rows[2], rows[3]);
      } else {
        s->rows[slot][lane] = rows[0];
      }
      const int live = SMALL ? 0 : __popc(__ballot_sync(0xffffffffu, rows[0] >= 0)) * run;
      if (lane == 0) s->live[slot] = f.valid ? live : -1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->rows_full[slot]);
      float sc[4];
#pragma unroll
      for (int i = 0; i < (SMALL ? 4 : 1); ++i) sc[i] = page[i] < 0 ? 0.0f : a.scale[page[i]];
      if constexpr (!SMALL) sc[0] = sc[1] = sc[2] = sc[3] = __shfl_sync(0xffffffffu, sc[0], 4 * lane / run);
      *reinterpret_cast<float4*>(&s->scale[slot][4 * lane]) = make_float4(sc[0], sc[1], sc[2], sc[3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->scale_full[slot]);
      if (++slot == SM::kAhead) { slot = 0; phase ^= 1u; }
    }
    if (!f.valid) return true;
  }
}

// Warp 0, pages of 8 rows and more: TMA boxes, half by half (half 0: the rotary entries and chunks 0, 1;
// half 1: chunks 2, 3) as P V frees them. One lane reads the rows, four at a time, and issues: boxes of
// 16 rows then take 30 cycles each. With a shuffle per row by the whole warp they took 80, and bound
// chunks of 33 queries on 128 heads in pages of 16: 153 us instead of 137.
template <int HG>
__device__ __forceinline__ bool lat_load_role(const LatAttnArgs& a, const CUtensorMap* tm_lat, const CUtensorMap* tm_rot,
                                              typename LatSmem<HG>::Info* s, uint8_t* smem) {
  using SM = LatSmem<HG>;
  volatile int* abort_flag = &s->abort;
  const bool leader = elect_one();
  const int run = a.run, pieces = kLatTile / run;
  const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
  const uint32_t bars = __shfl_sync(0xffffffffu, smem_u32(&s->kv_full[0]), 0);
  const uint64_t lat = reinterpret_cast<uint64_t>(tm_lat), rotary = reinterpret_cast<uint64_t>(tm_rot);
  for (int it = 0;; ++it) {
    const int ahead = it % SM::kAhead;
    if (!__all_sync(0xffffffffu, lat_wait(&s->rows_full[ahead], (it / SM::kAhead) & 1, abort_flag))) return false;
    const int live = __shfl_sync(0xffffffffu, s->live[ahead], 0);
    if (live < 0) return true;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const LatHalf h = lat_half<SM::kHalves>(2 * it + half);
      bool ok = lat_wait(&s->kv_empty[h.slot], h.phase ^ 1u, abort_flag);
      if (half == 0) ok = ok && lat_wait(&s->rot_empty[it % SM::kRots], ((it / SM::kRots) & 1) ^ 1u, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) return false;
      if (leader) {
        const uint32_t full = bars + h.slot * 8;
        uint32_t dst = base + h.slot * kLatHalf, rot = base + SM::kOffRot + it % SM::kRots * kLatRot;
        mbar_arrive_expect_tx(&s->kv_full[h.slot], live * (half == 0 ? 320 : 256));
#pragma unroll 1
        for (int i = 0; i < pieces; i += 4) {
          const int4 r4 = *reinterpret_cast<const int4*>(&s->rows[ahead][i]);
          const int r[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (r[k] >= 0) {
              tma_load_at(dst, lat, full, half * 256, r[k]);
              tma_load_at(dst + kLatChunk, lat, full, half * 256 + 128, r[k]);
              if (half == 0) tma_load_at(rot, rotary, full, 512, r[k]);
            }
            dst += run * 128;
            rot += run * 64;
          }
        }
        if (half == 1) mbar_arrive(&s->tab_empty[ahead]);
      }
      __syncwarp();
    }
  }
}

// Four warps, smaller pages: 16-byte asynchronous copies into the places (and the swizzle) that the
// boxes would use. A tile of single rows, copied alone from L2, takes 4500 cycles as TMA gathers from four warps
// and 3200 so. In the kernel a tile takes about 5000: 64 x 8192 tokens on 16 heads 85 us with a page each, 67 with
// pages of 64 by TMA (HBM needs 47). A warp copies 32 rows, each of its instructions 64 bytes of 8 rows, and
// has two halves in flight at most, of the five that the ring holds.
template <int HG>
__device__ __forceinline__ bool lat_copy_role(const LatAttnArgs& a, const uint8_t* cache, typename LatSmem<HG>::Info* s,
                                              uint8_t* smem) {
  using SM = LatSmem<HG>;
  volatile int* abort_flag = &s->abort;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const int r8 = lane >> 2, l4 = lane & 3;                 // row of 8, 16 bytes of 64
  const uint32_t in_tile = smem_u32(smem) + (warp * 32 + r8) * 128;
  const uint32_t lo = (l4 ^ r8) * 16, hi = ((4 + l4) ^ r8) * 16;       // the two 64-byte parts of a 128-byte row
  const uint32_t in_rot = smem_u32(smem) + SM::kOffRot + (warp * 32 + r8) * 64 + (l4 ^ ((r8 >> 1) & 3)) * 16;
  int pending = -1;                                        // slot whose copies have been issued but not announced
  auto announce = [&]() {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s->kv_full[pending]);
    pending = -1;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {        // announces what is pending before it has to wait
    if (__all_sync(0xffffffffu, mbar_test_at(smem_u32(bar), parity))) return true;
    if (pending >= 0) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      announce();
    }
    return __all_sync(0xffffffffu, lat_wait(bar, parity, abort_flag)) != 0;
  };
  bool ok = true;
  for (int it = 0; ok; ++it) {
    const int ahead = it % SM::kAhead;
    ok = wait(&s->rows_full[ahead], (it / SM::kAhead) & 1);
    if (!ok || s->live[ahead] < 0) break;
    const uint8_t* src[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int row = s->rows[ahead][warp * 32 + g * 8 + r8];
      src[g] = row < 0 ? nullptr : cache + static_cast<size_t>(row) * kLatDk + l4 * 16;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&s->tab_empty[ahead]);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const LatHalf h = lat_half<SM::kHalves>(2 * it + half);
      ok = wait(&s->kv_empty[h.slot], h.phase ^ 1u) &&
           (half == 1 || wait(&s->rot_empty[it % SM::kRots], ((it / SM::kRots) & 1) ^ 1u));
      if (!ok) break;
      const uint32_t dst = in_tile + h.slot * kLatHalf, rot = in_rot + it % SM::kRots * kLatRot;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (!src[g]) continue;
        const uint8_t* from = src[g] + half * 256;
        const uint32_t to = dst + g * 8 * 128;
        cp_async_16(to + lo, from);
        cp_async_16(to + hi, from + 64);
        cp_async_16(to + kLatChunk + lo, from + 128);
        cp_async_16(to + kLatChunk + hi, from + 192);
        if (half == 0) cp_async_16(rot + g * 8 * 64, src[g] + 512);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (pending >= 0) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        announce();
      }
      pending = h.slot;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (ok && pending >= 0) announce();
  return ok;
}

// ---------------------------------------------------------------- the kernel
// Registers a thread: 153 with 16 columns (128 for small pages); with 32, all that the threads' number leaves, 96
// and 56 bytes spilled (80 and 108 for small pages). 64 x 8192 tokens on 16 heads in pages of 64: 61.6 us in a
// graph, 0.75 of HBM over all; chunks of 500 queries 162 us, of which the MMAs alone need 83.
template <int HG, bool SMALL>
__global__ void __launch_bounds__(kLatThreads<HG, SMALL>, 1)
mla_fp8_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rot,
               const __grid_constant__ LatAttnArgs a) {
  using SM = LatSmem<HG>;
  constexpr int kThreads = kLatThreads<HG, SMALL>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  typename SM::Info* s = reinterpret_cast<typename SM::Info*>(smem + SM::kOffInfo);
  volatile int* abort_flag = &s->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kGroups = SM::kGroups;
  if (smem + SM::kUsed > smem_raw + SM::kBytes) {          // (an unaligned start of shared memory)
    if (threadIdx.x == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      raise_device_error(FP8MOE_DEVERR_TIMEOUT);
      a.merge[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    return;
  }

  if (warp == 0) {                                         // a lane per barrier
    if (lane < SM::kHalves) {
      mbar_init(&s->kv_full[lane], SMALL ? 4 : 1);
      mbar_init(&s->kv_empty[lane], 1);
    }
    if (lane < SM::kAhead) {
      mbar_init(&s->rows_full[lane], 1);
      mbar_init(&s->scale_full[lane], 1);
      mbar_init(&s->tab_empty[lane], (SMALL ? 4 : 1) + 4 * kGroups);
    }
    if (lane < 2) {
      mbar_init(&s->rot_empty[lane], 1);
      mbar_init(&s->s_full[lane], 1);
      mbar_init(&s->s_empty[lane], 4 * kGroups);
      mbar_init(&s->frag_full[lane], 1);
      mbar_init(&s->frag_empty[lane], 2 + 4 * kGroups);
    }
    if (lane < SM::kPBufs) {
      mbar_init(&s->p_full[lane], 4 * kGroups);
      mbar_init(&s->p_empty[lane], 1);
    }
    if (lane == 0) {
      mbar_init(&s->q_full, kGroups);
      s->abort = 0;
    }
    fence_mbar_init();
    if (!SMALL && lane == 0 && a.table.num_indices > 0) {  // (an empty table comes without maps)
      prefetch_tensormap(&tm_lat);
      prefetch_tensormap(&tm_rot);
    }
    __syncwarp();
  }
  if (warp == 2) {
    tmem_alloc(&s->tmem, SM::kTmemCols);
    tmem_relinquish();
  }
  // Launched while the work before it in the stream may still run: nothing above reads or writes what
  // that work does.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the work list's length, and the sequence that this CTA's share begins in: a run of
  // sequences per thread, then a scan over the threads
  const int per = (a.table.B + kThreads - 1) / kThreads;
  const int b0 = threadIdx.x * per, b1 = min(a.table.B, b0 + per);
  long long mine = 0;
  LatShape sh{};
  for (int b = b0; b < b1; ++b) {
    sh = lat_shape(a, b, HG);
    mine += static_cast<long long>(sh.groups) * sh.tiles;
  }
  long long incl = mine;
  for (int d = 1; d < 32; d <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += up;
  }
  // tiles of the longest sequence, if none has more than one column group
  const int most_here = static_cast<int>(
      __reduce_max_sync(0xffffffffu, per > 1 || sh.groups > 1 ? 0x7fffffffu : static_cast<unsigned>(sh.tiles)));
  if (lane == 31) {
    s->scan[warp] = incl;
    s->scan_most[warp] = most_here;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long before = incl - mine, total = 0;
  int most = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s->scan[w];
    total += s->scan[w];
    most = max(most, s->scan_most[w]);
  }
  const int gang_id = blockIdx.x >> a.gang_log, rank = blockIdx.x - (gang_id << a.gang_log);
  const int gangs = static_cast<int>(gridDim.x >> a.gang_log);
  // A sequence per gang, whole, where they are few and the longest has little more than an equal share:
  // a tile more costs less than a second fragment and joining. On 16 columns 2.9 tiles more gained 1.0
  // us (64 x 544 tokens: 15.8 instead of 16.8), 3.8 lost 2 (8 x 400); on 32, 2.5 gained four (30 x 700 on
  // 128 heads: 25 instead of 29).
  constexpr int kQuarters = HG == 16 ? 13 : 15;
  const bool whole = a.table.B <= gangs && (4ll * most - kQuarters) * gangs <= 4 * total;
  const int ngangs = static_cast<int>(min(static_cast<long long>(gangs), total));
  const long long p0 = lat_div(total * gang_id, max(ngangs, 1));
  const bool works = gang_id < (whole ? a.table.B : ngangs);
  if (whole) {
    if (static_cast<int>(threadIdx.x) == gang_id) {          // (without a sequence: an empty share)
      s->start_b = gang_id;
      s->start_off = before;
      s->start = sh;
    }
  } else if (works && p0 >= before && p0 < before + mine) {
    long long off = before;
    for (int b = b0; b < b1; ++b) {
      if (per > 1) sh = lat_shape(a, b, HG);
      const long long w = static_cast<long long>(sh.groups) * sh.tiles;
      if (p0 < off + w) {
        s->start_b = b;
        s->start_off = off;
        s->start = sh;
        break;
      }
      off += w;
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = s->tmem;
  bool ok = true;
  if (!works) {
    if (threadIdx.x == 0) a.merge[blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (SMALL && warp >= 4 + 4 * kGroups) {
    ok = lat_copy_role<HG>(a, a.cache, s, smem);
  } else if (warp == 2) {
    ok = lat_value_role<HG>(s, smem, tmem);
  } else if (warp >= 4) {
    ok = lat_softmax_role<HG>(a, s, smem, tmem);
  } else if (warp == 1) {
    ok = lat_score_role<HG>(s, smem, tmem);
  } else if (warp == 3) {
    const long long from = whole ? s->start_off : p0;
    const long long to = whole ? from + static_cast<long long>(s->start.groups) * s->start.tiles
                               : lat_div(total * (gang_id + 1), ngangs);
    LatSchedule<HG> schedule{s->start, s->start_b, s->start_off, from, from, to, total, ngangs, gang_id, rank,
                             make_int4(0, 0, 0, 0)};
    ok = lat_table_role<HG, SMALL>(a, s, schedule);
    if (!ok && lane == 0) a.merge[blockIdx.x] = make_int4(0, 0, 0, 0);   // the joining kernel must not find old words
  } else if constexpr (!SMALL) {
    ok = lat_load_role<HG>(a, &tm_lat, &tm_rot, s, smem);
    if (!ok) {
      // copies already in flight must land before the CTA's shared memory goes away
      const unsigned long long t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 10000000ull) {}
    }
  }
  if (!ok) {
    if (!*abort_flag) raise_device_error(FP8MOE_DEVERR_TIMEOUT);
    *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, SM::kTmemCols);
  }
}

// A weighted sum of parts under one reference (the largest is the least m), which moves as parts join.
template <int N>
struct LatSum {
  float m = kLatNoRef, l = 0.0f;
  float4 acc[N];
  __device__ __forceinline__ LatSum() {
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  __device__ __forceinline__ void add(const float2 ml, const float4 (&x)[N]) {
    if (ml.y == 0.0f) return;
    const float next = fminf(m, ml.x), w0 = exp2f(next - m), w1 = exp2f(next - ml.x);
    m = next;
    l = l * w0 + ml.y * w1;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      acc[j].x = acc[j].x * w0 + x[j].x * w1;
      acc[j].y = acc[j].y * w0 + x[j].y * w1;
      acc[j].z = acc[j].z * w0 + x[j].z * w1;
      acc[j].w = acc[j].w * w0 + x[j].w * w1;
    }
  }
  // values 4 i .. 4 i + 3 (i = at, at + step, ..) of output row `row`
  __device__ __forceinline__ void store(const LatAttnArgs& a, size_t row, int at, int step) const {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      __align__(8) const __nv_bfloat162 y[2] = {__floats2bfloat162_rn(acc[j].x * inv, acc[j].y * inv),
                                                __floats2bfloat162_rn(acc[j].z * inv, acc[j].w * inv)};
      reinterpret_cast<uint2*>(a.o + row * kLatDv)[at + j * step] = *reinterpret_cast<const uint2*>(y);
    }
    if (a.lse && at == 0) a.lse[row] = l == 0.0f ? -INFINITY : (log2f(l) - m) * 0.6931471805599453f;
  }
};

// Joins the parts of the column groups that were cut, in order, so the same bits every time. A part
// holds sums of 2^(score + m) and of those times values. blockIdx.x is the CTA that holds a first part.
// Up to eight parts: a warp per column, four columns a block. More (long contexts of few sequences):
// a block per column, eight parts' loads in flight; with a warp per column the 74 parts of two
// 128K-token sequences took 35 us more. Bound by three dependent reads from L2.
template <int HG>
__global__ void __launch_bounds__(128) mla_fp8_join_kernel(const LatAttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the parts are written
  const int cta = blockIdx.x;
  const int4 job = a.merge[cta];
  const int c = job.z <= 8 ? blockIdx.y * 4 + (threadIdx.x >> 5) : blockIdx.y;
  if (c >= job.y) return;                                  // (no columns: nothing to join)
  auto slot = [&](int i) { return static_cast<size_t>(i == 0 ? job.w : 2 * (cta + (i << a.gang_log))) * HG; };
  if (job.z <= 8) {
    const int lane = threadIdx.x & 31;
    LatSum<4> sum;
#pragma unroll 2
    for (int i = 0; i < job.z; ++i) {
      const size_t at = slot(i) + c;
      float4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = reinterpret_cast<const float4*>(a.part_o + at * kLatDv)[j * 32 + lane];
      sum.add(a.part_ml[at], x);
    }
    sum.store(a, static_cast<size_t>(job.x) + c, lane, 32);
    return;
  }
  LatSum<1> sum;
  constexpr int kBatch = 8;
  for (int i0 = 0; i0 < job.z; i0 += kBatch) {
    float2 ml[kBatch];
    float4 x[kBatch][1];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const size_t at = slot(min(i0 + k, job.z - 1)) + c;
      ml[k] = a.part_ml[at];
      if (i0 + k >= job.z) ml[k].y = 0.0f;
      x[k][0] = reinterpret_cast<const float4*>(a.part_o + at * kLatDv)[threadIdx.x];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) sum.add(ml[k], x[k]);
  }
  sum.store(a, static_cast<size_t>(job.x) + c, threadIdx.x, 128);
}

}  // namespace fp8moe
