// tree.cu — attention of drafted tokens over a paged cache (include/pi_draft.h).
#include <type_traits>

#include "serve.cuh"

namespace pis {

struct TreeArgs {
  const float *q, *k_new, *v_new;
  const int *parent, *count, *table, *len;
  uint16_t* pool;  // the layer's pages
  float *y, *lse;
  int* status;
  int slots, drafts, heads, kv_heads, group, head_dim, page_tokens, pages, max_pages, window, sinks;
  float scale;  // scale log2(e)
};

// What a slot's drafts see: the tokens [tail, base) and [0, first) before
// them, and one another.  The drafts begin at token base; the one of depth d (0
// without a parent) stands at position base + d, and a window hides from it the
// tokens below base + d + 1 - window but for the first `sinks`.
struct TreeSlot {
  int base, count, tail, first;
};
__device__ __forceinline__ TreeSlot tree_slot(const TreeArgs& a, int slot) {
  TreeSlot v;
  const int n = __ldg(a.len + slot), c = a.count ? __ldg(a.count + slot) : a.drafts;
  const bool ok = n >= 0 && n <= a.max_pages * a.page_tokens && c >= 0 && c <= a.drafts && c <= n;
  v.count = ok ? c : 0;
  v.base = ok ? n - c : 0;
  v.tail = a.window > 0 ? max(0, v.base + 1 - a.window) : 0;
  if (a.sinks >= v.tail) v.tail = 0;  // nothing in between
  v.first = min(v.tail, a.sinks);
  return v;
}
__device__ __forceinline__ bool tree_slot_bad(const TreeArgs& a, int slot) {
  const int n = __ldg(a.len + slot), c = a.count ? __ldg(a.count + slot) : a.drafts;
  return n < 0 || n > a.max_pages * a.page_tokens || c < 0 || c > a.drafts || c > n;
}

// The drafts that draft i sees, as bits: itself and its ancestors, in the
// window.  `parent(j)` gives a draft's parent; one that is not -1 .. j - 1
// counts as -1 (reported).
template <typename F>
__device__ __forceinline__ unsigned long long tree_path(const TreeArgs& a, int i, F parent) {
  unsigned long long path = 0;
  for (int j = i; j >= 0;) {
    path |= 1ull << j;
    int p = parent(j);
    if (p < -1 || p >= j) {
      set_status(a.status, PI_ERR_INDEX);
      p = -1;
    }
    j = p;
  }
  return path;
}
__device__ __forceinline__ unsigned long long tree_seen(const TreeArgs& a, int base, unsigned long long path) {
  const int hidden = a.window > 0 ? __popcll(path) - a.window : 0;  // the path's first ones
  unsigned long long seen = path;
  for (int d = 0; d < hidden; ++d) {  // the one of depth d
    const unsigned long long bit = path & -path;
    path ^= bit;
    if (base + d >= a.sinks) seen ^= bit;
  }
  return seen;
}

// A query row's sums over some of its tokens: the running maximum m of the
// scores (in base 2), l = sum 2^(a - m), o = sum 2^(a - m) v.
struct RowSums {
  float m, l;
  float o[8];  // of elements 8 lane + i
};

// Adds 32 tokens, one per lane, by the formulas in fp32 (any operand, infinite
// ones too).  `key`: the lane's key, null where its token is not seen; `val`:
// its value; fp32 rows (NEW) are taken as rounded to the cache's type.
template <int DT, bool NEW>
__device__ __forceinline__ void row_add32(const TreeArgs& a, const float* q, const void* key, const void* val,
                                          RowSums& r) {
  const int lane = threadIdx.x & 31, D = a.head_dim;
  auto piece = [](const void* row, int e, float (&x)[8]) {
    if (NEW) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(row) + (e >> 2));
      const float4 w = __ldg(reinterpret_cast<const float4*>(row) + (e >> 2) + 1);
      const float f[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = from_bits<DT>(to_bits<DT>(f[i]));
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(row) + e);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = from_bits<DT>((uint16_t)(w[i >> 1] >> 16 * (i & 1)));
    }
  };
  float s = -INFINITY;
  if (key) {
    s = 0.f;
    for (int e = 0; e < D; e += 8) {
      float k[8];
      piece(key, e, k);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(__ldg(q + e + i), k[i], s);
    }
    s *= a.scale;
  }
  float up = s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) up = fmaxf(up, __shfl_xor_sync(~0u, up, o));
  up = fmaxf(up, r.m);
  const float ref = up == -INFINITY ? 0.f : up;
  const float was = part_weight(r.m - ref), p = key ? ex2(s - ref) : 0.f;
  // an infinite value's weight is not 0 unless its score is -infinity
  const float w = key && s != -INFINITY ? fmaxf(p, 0x1p-126f) : p;
  r.m = up;
  r.l = fmaf(r.l, was, warp_sum(p));
#pragma unroll
  for (int i = 0; i < 8; ++i) r.o[i] *= was;
  for (uint32_t left = __ballot_sync(~0u, key != nullptr); left; left &= left - 1) {
    const int j = __ffs(left) - 1;
    const float wj = __shfl_sync(~0u, w, j);
    const void* row = reinterpret_cast<const void*>(
        __shfl_sync(~0u, reinterpret_cast<unsigned long long>(val), j));
    if (8 * lane < D) {
      float v[8];
      piece(row, 8 * lane, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) r.o[i] = fmaf(wj, v[i], r.o[i]);
    }
  }
}

// Adds the cached tokens [t0, t1), of which those at or past `lo` and the
// first `sinks` are seen.
template <int DT>
__device__ __forceinline__ void row_add_cached(const TreeArgs& a, int slot, int g, const float* q, int t0, int t1,
                                               int lo, RowSums& r, int* beat) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (unsigned at = 0; (int)at >= 0 && (int)at < t1 - t0; at += 32) {
    const int t = t0 + (int)min(at + lane, (unsigned)(t1 - t0 - 1));
    if (lane == 0) atomicAdd(beat, 1);
    const uint16_t* key = nullptr;
    if (at + lane < (unsigned)(t1 - t0) && (t >= lo || t < a.sinks)) {
      const int j = t / a.page_tokens;
      const int page = checked_page(__ldg(a.table + (size_t)slot * a.max_pages + j), a.pages, a.status);
      if (page >= 0)
        key = a.pool + (((size_t)page * 2 * a.kv_heads + g) * a.page_tokens + t - j * a.page_tokens) * a.head_dim;
    }
    row_add32<DT, false>(a, q, key, key + (size_t)a.kv_heads * a.page_tokens * a.head_dim, r);
  }
}

// Adds the drafts `seen`.
template <int DT>
__device__ __forceinline__ void row_add_drafts(const TreeArgs& a, int slot, const TreeSlot& v, int g, const float* q,
                                               unsigned long long seen, RowSums& r) {
  const int lane = threadIdx.x & 31;
  if (!a.k_new) {
    for (int j0 = 0; j0 < v.count; j0 += 32) {
      const int t = v.base + j0 + lane;
      const uint16_t* key = nullptr;
      if (j0 + lane < v.count && seen >> (j0 + lane) & 1) {
        const int j = t / a.page_tokens;
        const int page = checked_page(__ldg(a.table + (size_t)slot * a.max_pages + j), a.pages, a.status);
        if (page >= 0)
          key = a.pool + (((size_t)page * 2 * a.kv_heads + g) * a.page_tokens + t - j * a.page_tokens) * a.head_dim;
      }
      row_add32<DT, false>(a, q, key, key + (size_t)a.kv_heads * a.page_tokens * a.head_dim, r);
    }
    return;
  }
  for (int j0 = 0; j0 < v.count; j0 += 32) {
    const bool ok = j0 + lane < v.count && seen >> (j0 + lane) & 1;
    const size_t row = (((size_t)slot * a.drafts + min(j0 + lane, v.count - 1)) * a.kv_heads + g) * a.head_dim;
    row_add32<DT, true>(a, q, ok ? a.k_new + row : nullptr, a.v_new + row, r);
  }
}

// ------------------------------------------------------------------ tensor cores
//
// Mathematics.  A query row's visible tokens may be split into any parts; part i
// yields m_i = max a_t, l_i = sum exp(a_t - m_i), o_i = sum exp(a_t - m_i) v_t, and
// parts join with the weights exp(m_i - max m).
//
// The query rows of a kv head are drafts x heads of its group.  Both products run
// on the fifth-generation tensor cores, operands in shared memory by TMA, sums in
// tensor memory, in one of two forms.
//   Many rows (MR = 128; 64 for head dimensions past 128): S = Q K^T has the rows as
//   the 128 rows of the product's tile and the tokens as its columns; a thread has a
//   row of S, so maxima and sums are its own, and the weights return to the place of
//   the scores that they come from, from where the second product O = P V reads them.
//   Few rows (MR = 16, 32): S^T = K Q^T has the tokens as rows and query rows x parts as
//   columns, a thread a token; O^T = V^T P^T, P through shared memory.  A tile then
//   costs 16 instructions of 32 to 96 columns instead of 32 to 48 of 128, and all threads
//   work whatever the number of rows.
// 32 slots x 40 heads of 128, 13 drafts (13 rows), lengths to 2048, fp16: 183 us, in the
// form of many rows 380.  The border: 16 slots, 32/8 heads of 128, 8001 tokens at most,
// fp16 (bf16), with 24 rows 74 us (75) against 87 (108) in the form of many rows, with 32
// 77 (78) against 85 (109); with 36 rows 87 (107) against 116 (118) as two units of 32, with
// 64 92 (114) against 123 (124), with 128 114 (137) against 241 (244) as four.
//
// A unit is (slot, kv head, MR query rows, up to 128 columns of V).  It goes
// through tiles of TN tokens: the drafts' own, then those of the cache.  The
// units' tiles, each unit preceded by tree_cost() positions for its fixed cost,
// form one line of which every block (one per SM: shared memory) takes an equal
// contiguous share; a unit that several blocks share is joined by a second kernel.
//
// Precision.  q and the weights p are fp32 and enter as sums of 16-bit parts (two
// in fp16, with q scaled by a power of two per row and p by 2^14; three in bf16),
// low parts first or in columns of their own.  A tile's O is read back and added to
// fp32 registers with a rounded add: the tensor cores' own sums would drift over a
// long cache.
//
// Roles of a block's warps.  0-7: load Q, softmax, and add up O: warps w and w + 4
// share the rows (few rows: the tokens) and halve the columns.  8: issues the MMAs, S
// of the next tile, then O of the last, so that the products run while the warps 0-7
// are at the tile in between.  From 9 on: fill K, or V: whole boxes of tokens by TMA,
// everything else (drafts, the ends of what is seen, odd page sizes) by hand, with zeros
// for values nobody sees.  New drafts' rows never come from the cache: no block waits for
// another's store.
//
// Bound.  Few rows: HBM, beside a unit's start and end (some 10000 cycles against 2800
// a tile, in series with them): 55 % of a copy's rate at 32 slots x 40 heads.  Many rows:
// the softmax warps, some 4200 cycles a tile of 128 rows x 128 tokens against 2200 of the
// products.  They issue in 38 % of the cycles and wait for tensor memory in most others:
// 32 columns are loaded and waited for at a time, twice.  8 slots, 64/8 heads, chains of 64
// (512 rows), lengths to 32768, fp16: 489 us, 520 TFLOP/s of the formula's operations, 1.0
// PFLOP/s as executed.  With 33 to 64 rows half of those warps have no rows, and head
// dimensions past 128 compute S and the weights once per half of V's columns.
// Pages that are no multiple of 8 tokens and head dimensions below 64 have no boxes: all
// rows by hand, a 16-byte load per thread and piece, 9 times as long (16 slots, 32/8 heads
// of 128, 13 drafts, 4096 tokens, fp16: 73 us with pages of 16, 76 with 24, 678 with 7).
//
// Operands that are not finite.  Rows whose sums come out NaN or infinite are
// gone through again in fp32, token by token, by the warp that would write them.
template <int DT, int DP, int MR>
struct TreeTile {  // MR: query rows of a unit
  static constexpr bool kFew = MR <= 32;
  static constexpr int KW = MR == 16 ? 2 : 1, VW = 2;  // warps that fill K, V
  static constexpr int kThreads = 32 * (9 + KW + VW);
  static constexpr int TN = DP == 256 ? 64 : 128;  // tokens of a tile
  static constexpr int DV = DP < 128 ? DP : 128;   // columns of V of a unit
  static constexpr int NP = DT == 0 ? 2 : 3;       // parts of q and p
  static constexpr int NQ = NP * MR;               // few rows: columns of S and O
  // stages of K, of V
  static constexpr int SV = DP == 64 ? 4 : DP == 256 && DT == 0 ? 3 : 2,
                       SK = kFew && DP == 128 && (DT == 0 || MR == 16) ? 3 : SV;
  static constexpr int NO = !kFew && DT == 1 && DP == 128 ? 1 : 2;  // O tiles in tensor memory
  static constexpr int kK = TN * DP * 2, kV = TN * DV * 2;  // bytes of a stage
  static constexpr int kQ = MR * DP * 2;                    // of a part of Q
  static constexpr int kP = kFew ? (NQ + 63) / 64 * TN * 128 : 0;  // of P, two of which
  static constexpr int kStages = (NP * kQ + 1023) / 1024 * 1024, kWeights = kStages + SK * kK + SV * kV,
                       kMisc = kWeights + 2 * kP, kValues = kStages + SK * kK;
  // tensor-memory columns.  Many rows: two S tiles, 16 columns of which become the
  // first two parts of P for the same 16 tokens; the third parts of P; O.  Few rows: two
  // S tiles; O.
  static constexpr int kS = kFew ? NQ : TN, kO1 = kFew ? NQ : DV;  // of a tile
  static constexpr int kThird = 2 * kS, kO = kThird + (!kFew && DT == 1 ? TN : 0);
  static_assert(kO + NO * kO1 <= 512, "tensor memory");
};
constexpr int kTreeWarps = 13;   // at most
constexpr int kTreeGrid = 192;   // most blocks
// A unit's fixed cost, in tiles: Q, its drafts' rows, its output.  A slot with nothing
// before its drafts is all fixed cost.  Measured at 32 slots x 40 heads, 13 drafts / 16
// slots, 32/8 heads, 6 drafts / 32 drafts / 8 slots, 64/8 heads, chains of 64, fp16: 186 /
// 74 / 114 / 488 us; with 2 for 4 188 / 82 / 110 / 487, with 6 191 / 76 / 116 / 496; drafts / 4
// for few rows 197, drafts / 8 for many 109 / 536, without the slope 145 / 950.  Rows by hand
// (odd pages, small heads) cost more than this; they have no rule of their own.
__host__ __device__ __forceinline__ int tree_cost(int mr, int drafts) { return 4 + (mr <= 32 ? drafts / 8 : drafts / 4); }
// Units of at most this many tiles are not split: one slot, 16 heads, 200 tokens 16.1 us
// (split 21.4), 64 slots, 32/8 heads, to 600 tokens 70.7 (80.8); with 12 one slot of 700
// tokens takes 26.6 for 23.6, 24 slots x 16 heads to 1000 tokens 47 for 52.
constexpr int kTreeWhole = 6;
// Least share of a block: one slot, 32/8 heads, 2048 tokens 25.3 us; with 1 29.7, with 6
// 27.6 (700 tokens: 23.6 and 28.7).
constexpr int kTreeShare = 3;
constexpr int kTreeHide = 8;     // more than the tiles between the filling of K and the softmax

// `total` positions over `blocks` blocks: the first `more` take one more.
struct TreeLine {
  long long each;
  int more;
  __device__ __forceinline__ void set(long long total, int blocks) {
    each = quotient(total, blocks);
    more = (int)(total - each * blocks);
  }
  __device__ __forceinline__ long long start(int b) const { return b * each + min(b, more); }
  __device__ __forceinline__ int block_of(long long pos) const {
    const long long head = more * (each + 1);
    return pos >= head ? more + (int)((pos - head) / each) : (int)(pos / (each + 1));
  }
};

struct TreeShared {
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4], sfull[2], pfull[2], ofull[2], oempty[2];
  uint64_t pair[4], qfull, fin;
  uint32_t taddr;
  int bad;
  int beat;  // goes on while rows are gone through again, which others wait for
  TreeLine line;
  long long share0;
  uint32_t hide[kTreeHide][4];  // tokens of a tile whose page is out of range
  union {
    float top[2][2][128];  // rows' maxima, of a tile's two halves; at a segment's end their sums
    float few[2][2][4][16];  // few rows: [..][half of the rows][32 tokens][row]
    struct {
      long long sum[kTreeWarps], len[kTreeWarps];
      int most[kTreeWarps];
      long long at;
      int slot, unit;
    } scan;
  };
};
struct TreeSharedScale : TreeShared {
  float qs[2][128];  // rows' 2^-e of q (fp16)
};
struct TreeSharedFew : TreeShared {  // of a segment's rows
  float4 figures[8][16];  // a warp's rows: factor of the scores, reference, the sums' factors
  float qs[2][32];
  int lo[2][32];
  u64 seen[2][32];
};
template <int DT, bool FEW>
using TreeSharedOf = std::conditional_t<FEW, TreeSharedFew, std::conditional_t<DT == 0, TreeSharedScale, TreeShared>>;
template <int DT, int DP, int MR>
__host__ __device__ constexpr int tree_smem() {
  return TreeTile<DT, DP, MR>::kMisc + (int)sizeof(TreeSharedOf<DT, MR <= 32>);
}

struct TreeSpan {  // a unit that begins in a block and ends in a later one
  int slot, unit, last, some;
};
struct TreeWork {
  TreeArgs a;
  TreeSpan* span;  // [grid]
  float* part;     // [grid][2][MR][DV + 4]
  int halves;      // units of V's columns
  int tma;         // tiles come as TMA boxes
  int box, edge;   // rows of a box: in tiles that are seen whole, in others
  int align;       // tokens that a window's first tile begins at a multiple of
  int page_shift;  // log2(page_tokens), or -1
  unsigned long long limit_ns;
  int lose;        // self-test: a copy is awaited that is never ordered
};

// More bytes of the phase under way, without an arrival.
__device__ __forceinline__ void mbar_expect_more(uint64_t* m, unsigned bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(m)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* m) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(m)) : "memory");
}
__device__ __forceinline__ void tree_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* m) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(m))
      : "memory");
}
// Shared-memory matrix descriptor, 128-byte swizzle.  K-major: sbo = the distance of
// 8-row groups.  MN-major: lbo = the distance of 64-element groups along M or N, sbo
// = that of 8-row groups along K.
__device__ __forceinline__ uint64_t tree_desc(uint32_t saddr, uint32_t lbo) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version of this family
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}
// Instruction descriptor of kind::f16: D fp32, A and B of DT, M = 128, N = n; A and B
// K-major, or M- and N-major.
template <int DT>
__device__ __forceinline__ uint32_t tree_idesc(int n, bool b_nmajor, bool a_mmajor = false) {
  return (1u << 4) | ((uint32_t)DT << 7) | ((uint32_t)DT << 10) | (a_mmajor ? 1u << 15 : 0u) | (b_nmajor ? 1u << 16 : 0u) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// True in one lane of the warp, the same one every time.
__device__ __forceinline__ bool elected() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* m) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(m))
               : "memory");
}
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The values of the loads before it may be used behind it.
template <int N>
__device__ __forceinline__ void tm_wait_ld(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_ld32(float* v, uint32_t t) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
__device__ __forceinline__ void tm_ld8(float* v, uint32_t t) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
__device__ __forceinline__ void tm_ld16(float* v, uint32_t t) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t));
}
__device__ __forceinline__ void tm_st8(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Two fp32 values rounded to 16 bits in one instruction (two conversions take four
// times as long as the packed one), and what that left.
template <int DT>
__device__ __forceinline__ uint32_t round2(float x, float y) {
  uint32_t r;
  if (DT == 0) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
template <int DT>
__device__ __forceinline__ u64 left2(u64 v, uint32_t r) {
  float2 h;
  if (DT == 0) h = __half22float2(*reinterpret_cast<const __half2*>(&r));
  else h = make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  return fma2(pair(h.x, h.y), pair(-1.f, -1.f), v);
}
// e for which 2^e takes a row's largest |q| into [2^13, 2^14); 126 at most, so that 2^-e is
// no subnormal, and 0 where it is 0 or not finite.
__device__ __forceinline__ int query_exponent(float top) {
  return top > 0.f && top < INFINITY ? 140 - max(14, (int)(__float_as_uint(top) >> 23)) : 0;
}
// The rows' values of all lanes joined, N rows: row i's in the lanes 32 i / N and on.
// Halves of the rows change places as halves of the lanes do.
template <int N, typename F>
__device__ __forceinline__ float warp_rows(float (&v)[N], F join) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = N / 2, off = 16; half >= 1; half >>= 1, off >>= 1) {
    const bool upper = lane & off;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
      v[i] = join(keep, __shfl_xor_sync(~0u, send, off));
    }
  }
#pragma unroll
  for (int off = 16 / N; off > 0; off >>= 1) v[0] = join(v[0], __shfl_xor_sync(~0u, v[0], off));
  return v[0];
}

// A unit and its tiles.
struct TreeUnit {
  int slot, unit;  // number within the slot: (g, rt, half)
  TreeSlot v;
  int g, row0, rows, half;  // query rows [row0, row0 + rows) of the kv head
  int start, firsts, tiles; // first token of the window's tiles; tiles of the first tokens; all
};
template <int TN>
__device__ __forceinline__ int tree_tiles(const TreeWork& w, const TreeSlot& v) {
  // lengths up to 2^31 - 1: nothing is added that could pass them
  const int start = v.tail & -w.align;
  return 1 + (v.first ? (v.first - 1) / TN + 1 : 0) + (v.base > v.tail ? (v.base - start - 1) / TN + 1 : 0);
}
__device__ __forceinline__ int tree_units(const TreeWork& w, const TreeSlot& v, int mr) {
  return v.count ? w.a.kv_heads * ((v.count * w.a.group + mr - 1) / mr) * w.halves : 0;
}
// Goes through a block's share: segments [tile0, tile1) of units.
template <int TN, int MR>
struct TreeWalk {
  const TreeWork& w;
  TreeUnit u;
  long long at, end;  // from the share's begin: of the unit on the line, of the share's end
  bool whole;
  int units;          // of the slot
  int tile0, tile1;
  __device__ __forceinline__ TreeWalk(const TreeWork& w, int slot, int unit, long long at, long long end, bool whole)
      : w(w), at(at), end(end), whole(whole) {
    u.slot = slot;
    u.unit = unit;
    if (at < end) open();
  }
  __device__ __forceinline__ void open() {
    u.v = tree_slot(w.a, u.slot);
    units = tree_units(w, u.v, MR);
    u.start = u.v.tail & -w.align;
    u.firsts = u.v.first ? (u.v.first - 1) / TN + 1 : 0;
    u.tiles = tree_tiles<TN>(w, u.v);
    fit();
  }
  __device__ __forceinline__ void fit() {
    const int rts = units / (w.a.kv_heads * w.halves), per = rts * w.halves;
    u.g = u.unit / per;
    const int r = u.unit - u.g * per, rt = r / w.halves;
    u.half = r - rt * w.halves;
    u.row0 = rt * MR;
    u.rows = min(MR, u.v.count * w.a.group - u.row0);
    if (whole) {
      tile0 = 0;
      tile1 = u.tiles;
    } else {
      const long long a1 = end - at - tree_cost(MR, u.v.count);
      tile0 = at < -tree_cost(MR, u.v.count) ? (int)(-at - tree_cost(MR, u.v.count)) : 0;
      tile1 = a1 < u.tiles ? (int)a1 : u.tiles;
    }
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ __forceinline__ bool any() const { return tile1 > tile0; }
  __device__ __forceinline__ bool begins() const { return tile0 == 0; }
  __device__ __forceinline__ bool ends() const { return tile1 == u.tiles; }
  __device__ __forceinline__ void next() {
    at += whole ? 1 : u.tiles + tree_cost(MR, u.v.count);
    if (at >= end) return;
    if (++u.unit < units) {
      fit();
      return;
    }
    u.unit = 0;
    do ++u.slot;
    while (u.slot < w.a.slots && tree_slot(w.a, u.slot).count == 0);
    if (u.slot >= w.a.slots) {
      at = end;
      return;
    }
    open();
  }
  // Tile i >= 1 holds the tokens from t0 on, of which [lo, hi) are seen by some draft.
  __device__ __forceinline__ int cached(int i, int& lo, int& hi) const {
    const bool first = i <= u.firsts;
    const int t0 = first ? (i - 1) * TN : u.start + (i - 1 - u.firsts) * TN;
    lo = first ? 0 : u.v.tail;
    hi = first ? u.v.first : u.v.base;
    return t0;
  }
  // Its columns in the products.
  __device__ __forceinline__ int columns(int i) const {
    if (i == 0) return (u.v.count + 15) & ~15;
    int lo, hi;
    const int t0 = cached(i, lo, hi);
    return (min(TN, hi - t0) + 15) & ~15;
  }
};

// A row's draft, and what it sees.
struct TreeRow {
  int draft, lo;  // lo: least visible cached token but for the first `sinks`
  unsigned long long seen;
  const float* q;
  size_t out;     // row of y
};
template <typename F>
__device__ __forceinline__ TreeRow tree_row(const TreeArgs& a, const TreeUnit& u, int r, F parent) {
  TreeRow x;
  const int R = u.row0 + r;
  x.draft = R / a.group;
  const unsigned long long path =
      a.parent ? tree_path(a, x.draft, parent) : (2ull << x.draft) - 1;
  x.lo = a.window > 0 ? u.v.base + __popcll(path) - a.window : 0;
  x.seen = tree_seen(a, u.v.base, path);
  x.out = ((size_t)u.slot * a.drafts + x.draft) * a.heads + u.g * a.group + R - x.draft * a.group;
  x.q = a.q + x.out * a.head_dim;
  return x;
}

// The segment [tile0, tile1) of row r once more, in fp32; the warp's lanes hold the
// columns 8 lane .. of it.
template <int DT, int TN, int MR>
__device__ __forceinline__ RowSums tree_again(const TreeWork& w, const TreeUnit& u, int tile0, int tile1, int r, int* beat) {
  const TreeArgs& a = w.a;
  const TreeRow x = tree_row(a, u, r, [&](int j) { return __ldg(a.parent + (size_t)u.slot * a.drafts + j); });
  RowSums s = {-INFINITY, 0.f, {}};
  const int f0 = max(tile0, 1) - 1, f1 = min(tile1 - 1, u.firsts);
  if (f0 < f1) row_add_cached<DT>(a, u.slot, u.g, x.q, f0 * TN, f1 == u.firsts ? u.v.first : f1 * TN, x.lo, s, beat);
  const int w0 = max(tile0 - 1 - u.firsts, 0), w1 = tile1 - 1 - u.firsts;
  if (w0 < w1)
    row_add_cached<DT>(a, u.slot, u.g, x.q, max(u.v.tail, u.start + w0 * TN),
                       tile1 == u.tiles ? u.v.base : u.start + w1 * TN, x.lo, s, beat);
  if (tile0 == 0) row_add_drafts<DT>(a, u.slot, u.v, u.g, x.q, x.seen, s);
  return s;
}

template <int DT, int DP, int MR>
__global__ void __launch_bounds__(TreeTile<DT, DP, MR>::kThreads, 1)
    tree_kernel(const __grid_constant__ TreeWork w, const __grid_constant__ CUtensorMap map,
                const __grid_constant__ CUtensorMap edge_map) {
  using C = TreeTile<DT, DP, MR>;
  constexpr bool kFew = C::kFew;
  constexpr int TN = C::TN, DV = C::DV, NP = C::NP, NQ = C::NQ, SK = C::SK, SV = C::SV, NO = C::NO;
  constexpr int kPanelK = TN * 128, kPanelQ = (kFew ? NQ : MR) * 128;  // bytes of 64 columns
  using Shared = TreeSharedOf<DT, kFew>;
  extern __shared__ __align__(1024) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::kMisc);
  const TreeArgs& a = w.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = a.head_dim, P = a.page_tokens;
  pdl_enter();

  // ---- the block's share of the line
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.kfull[i], C::KW);
      mbar_init(&sh.vfull[i], C::VW);
      mbar_init(&sh.kempty[i], 1);
      mbar_init(&sh.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.pfull[i], 8);
      mbar_init(&sh.ofull[i], 1);
      mbar_init(&sh.oempty[i], 8);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.pair[i], kFew ? 4 : 2);
    mbar_init(&sh.qfull, 8);
    mbar_init(&sh.fin, 1);
    fence_mbar_init();
    sh.bad = sh.beat = 0;
    w.span[blockIdx.x] = TreeSpan{0, 0, 0, 0};
  }
  long long share0, share1, unit_at;
  int first_slot, first_unit, grid;
  bool whole;
  TreeLine line;
  {
    auto& sc = sh.scan;
    const int k = (a.slots + C::kThreads - 1) / C::kThreads, s0 = tid * k, s1 = min(a.slots, s0 + k);
    long long units = 0, tiles = 0;
    int most = 0;
    for (int s = s0; s < s1; ++s) {
      const TreeSlot v = tree_slot(a, s);
      if (blockIdx.x == 0 && tree_slot_bad(a, s)) set_status(a.status, PI_ERR_INDEX);
      const int n = tree_units(w, v, MR), t = tree_tiles<TN>(w, v);
      units += n;
      tiles += (long long)n * (t + tree_cost(MR, v.count));
      if (n) most = max(most, t);
    }
    auto sum_up = [&](long long v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += x;
      }
      return v;
    };
    const long long upto_u = sum_up(units), upto_t = sum_up(tiles);
    most = (int)__reduce_max_sync(~0u, (uint32_t)most);
    if (lane == 31) {
      sc.sum[warp] = upto_u;
      sc.len[warp] = upto_t;
    }
    if (lane == 0) sc.most[warp] = most;
    __syncthreads();
    long long all_u = 0, all_t = 0, low_u = 0, low_t = 0;
    most = 0;
    for (int i = 0; i < C::kThreads / 32; ++i) {
      if (i == warp) low_u = all_u, low_t = all_t;
      all_u += sc.sum[i];
      all_t += sc.len[i];
      most = max(most, sc.most[i]);
    }
    whole = most <= kTreeWhole;
    const long long total = whole ? all_u : all_t;
    grid = gridDim.x;
    const long long useful = whole ? all_u : max(1ll, all_t / kTreeShare);
    if (useful < grid) grid = max(1, (int)useful);
    line.set(total, grid);
    share0 = share1 = 0;
    if ((int)blockIdx.x < grid) {
      share0 = line.start(blockIdx.x);
      share1 = line.start(blockIdx.x + 1);
    }
    // the thread whose slots hold the share's start
    long long at = whole ? low_u + upto_u - units : low_t + upto_t - tiles;
    if (share0 >= at && share0 < at + (whole ? units : tiles) && share0 < share1) {
      for (int s = s0; s < s1; ++s) {
        const TreeSlot v = tree_slot(a, s);
        const int n = tree_units(w, v, MR), len = whole ? 1 : tree_tiles<TN>(w, v) + tree_cost(MR, v.count);
        if (share0 < at + (long long)n * len) {
          sc.slot = s;
          sc.unit = (int)((share0 - at) / len);
          sc.at = at + (long long)sc.unit * len;
          break;
        }
        at += (long long)n * len;
      }
    }
    __syncthreads();
    const bool some = share0 < share1;
    if (tid == 0) {
      sh.line = line;
      sh.share0 = share0;
    }
    first_slot = some ? sc.slot : 0;
    first_unit = some ? sc.unit : 0;
    unit_at = some ? sc.at : 0;
    if (warp == 8) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.taddr)));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
  }
  const uint32_t tmem = sh.taddr;
  TreeWalk<TN, MR> walk(w, first_slot, first_unit, unit_at - share0, share1 - share0, whole);
  const int kd = (D + 15) >> 4;  // steps of 16 along a row
  int t = 0;                     // tiles so far
  bool ok = true;
  auto gave_up = [&] {
    set_status(a.status, PI_ERR_TIMEOUT);
    *(volatile int*)&sh.bad = 1;
    ok = false;
  };
  // A bounded wait, begun anew while rows are gone through again.
  auto wait_for = [&](uint64_t* bar, uint32_t parity) {
    for (;;) {
      const int beat = __shfl_sync(~0u, *(volatile int*)&sh.beat, 0);
      if (mbar_wait(bar, parity, w.limit_ns)) return true;
      if (__shfl_sync(~0u, *(volatile int*)&sh.beat, 0) == beat) return false;
    }
  };
#define TREE_WAIT(bar, parity)              \
  if (!wait_for(bar, (uint32_t)(parity))) { \
    gave_up();                              \
    break;                                  \
  }

  if (warp < 8) {
    if constexpr (!kFew) {
    // ---- Q, softmax, O
    constexpr int HC = TN / 2, HO = DV / 2;  // a half's columns of S, of O
    const int h = warp >> 2, wq = warp & 3, row = 32 * wq + lane;
    const float flip = a.scale < 0.f ? -1.f : a.scale == 0.f ? 0.f : 1.f;
    const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale);
    constexpr float kShift = DT == 0 ? 14.f : 0.f;
    const uint32_t lanes = tmem + ((uint32_t)(32 * wq) << 16);
    int seg = 0, met = 0;
    // The other half's value of the row; false where the wait ran out.
    auto meet = [&](float mine, float& theirs) {
      sh.top[met & 1][h][row] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.pair[wq]);
      if (!mbar_spin(&sh.pair[wq], (uint32_t)(met & 1)) && !wait_for(&sh.pair[wq], (uint32_t)(met & 1))) return false;
      theirs = sh.top[met & 1][1 - h][row];
      ++met;
      return true;
    };
    for (; walk.more() && ok; walk.next()) {
      if (!walk.any()) continue;
      const TreeUnit& u = walk.u;
      // rows warp, warp + 8, ...: split into parts
      constexpr int E = DP / 32, B = DP == 256 ? 4 : 8;
#pragma unroll 1
      for (int r0 = warp; r0 < u.rows; r0 += 8 * B) {
        float x[B][E];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int r = r0 + 8 * b;
          const int R = u.row0 + r, i = R / a.group;
          const float* q = a.q + (((size_t)u.slot * a.drafts + i) * a.heads + u.g * a.group + R - i * a.group) * D + E * lane;
          if (r < u.rows && E * lane < D) {
            if constexpr (E == 2) {
              const float2 f = __ldg(reinterpret_cast<const float2*>(q));
              x[b][0] = f.x, x[b][1] = f.y;
            } else {
#pragma unroll
              for (int e = 0; e < E; e += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(q + e));
                x[b][e] = f.x, x[b][e + 1] = f.y, x[b][e + 2] = f.z, x[b][e + 3] = f.w;
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[b][e] = 0.f;
          }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int r = r0 + 8 * b;
          if (r >= u.rows) break;
          if constexpr (DT == 0) {
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(x[b][e]));
            top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));
            const int ex = query_exponent(top);
            const float f = __uint_as_float((uint32_t)(ex + 127) << 23);
#pragma unroll
            for (int e = 0; e < E; ++e) x[b][e] *= f;
            if (lane == 0) sh.qs[seg & 1][r] = __uint_as_float((uint32_t)(127 - ex) << 23);
          }
          uint32_t part[NP][E / 2];
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            float y = x[b][2 * e] * flip, z = x[b][2 * e + 1] * flip;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              part[p][e] = pack_bits<DT>(y, z);
              y -= from_bits<DT>((uint16_t)part[p][e]);
              z -= from_bits<DT>((uint16_t)(part[p][e] >> 16));
            }
          }
          const int c = E * lane;
          unsigned char* to = smem + (c >> 6) * kPanelQ + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4) + 2 * (c & 7);
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            if constexpr (E == 2) *reinterpret_cast<uint32_t*>(to + p * C::kQ) = part[p][0];
            else if constexpr (E == 4) *reinterpret_cast<uint2*>(to + p * C::kQ) = make_uint2(part[p][0], part[p][1]);
            else *reinterpret_cast<uint4*>(to + p * C::kQ) = make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
          }
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.qfull);
      // the row's own draft
      const bool live = 32 * wq < u.rows;
      int pa = -1, pb = -1;
      if (live && a.parent) {
        if (lane < u.v.count) pa = __ldg(a.parent + (size_t)u.slot * a.drafts + lane);
        if (lane + 32 < u.v.count) pb = __ldg(a.parent + (size_t)u.slot * a.drafts + lane + 32);
      }
      int lo = 0;
      unsigned long long seen = 0;
      if (live) {
        const int draft = (u.row0 + min(row, u.rows - 1)) / a.group;
        unsigned long long path = (2ull << draft) - 1;
        if (a.parent) {  // all lanes together: the parents are in their registers
          path = 0;
          int j = draft;
          while (__any_sync(~0u, j >= 0)) {
            const int x0 = __shfl_sync(~0u, pa, j & 31), x1 = __shfl_sync(~0u, pb, j & 31);
            if (j >= 0) {
              path |= 1ull << j;
              int p = j < 32 ? x0 : x1;
              if (p < -1 || p >= j) {
                set_status(a.status, PI_ERR_INDEX);
                p = -1;
              }
              j = p;
            }
          }
        }
        lo = a.window > 0 ? u.v.base + __popcll(path) - a.window : 0;
        seen = tree_seen(a, u.v.base, path);
      }
      TREE_WAIT(&sh.qfull, seg & 1);
      float scl = scale;
      if constexpr (DT == 0) scl = live && row < u.rows ? scale * sh.qs[seg & 1][row] : scale;
      ++seg;
      const int sinks = u.v.tail > 0 ? 0 : a.sinks;
      float m = -INFINITY, ref = -INFINITY, l = 0.f, alpha = 0.f;
      const int first = h * HC;  // column
      u64 o2[HO / 2];
#pragma unroll
      for (int c = 0; c < HO / 2; ++c) o2[c] = 0;
      for (int i = walk.tile0;; ++i, ++t) {  // the softmax of tile i, then the sums with tile i - 1's O
        const int buf = t & 1;
        const float before = alpha;
        const bool tile = i < walk.tile1;
        if (tile) TREE_WAIT(&sh.sfull[buf], (t >> 1) & 1);
        if (live && tile) {
          tm_fence_after();
          const uint32_t src = lanes + (uint32_t)(buf * TN + first);
          // the columns that the row does not see, 16 at a time
          int any_lo = 0, hi = 0, t0 = 0;
          if (i > 0) t0 = walk.cached(i, any_lo, hi);
          const int from = i <= u.firsts ? 0 : lo;
          bool all = i > 0 && t0 >= from && hi - t0 >= TN;
#pragma unroll
          for (int k = 0; k < TN / 32; ++k) all &= !sh.hide[t % kTreeHide][k];
          all = __all_sync(~0u, all);
          auto hide = [&](int k, float* v) {  // of the 16 columns k
            auto below = [](int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1u; };
            const int c0 = first + 16 * k, at = t0 + c0;
            uint32_t mask = i > 0 ? below(hi - at) & (~below(from - at) | below(sinks - at))
                                  : c0 < 64 ? (uint32_t)(seen >> c0) : 0u;
            mask &= ~(sh.hide[t % kTreeHide][c0 >> 5] >> (c0 & 31));
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] = mask >> c & 1u ? v[c] : -INFINITY;
          };
          float top = -INFINITY, theirs = 0.f;
          auto top_of = [&](int k) {  // of 32 columns from 16 k on
            float v[32];
            tm_ld32(v, src + 16 * k);
            tm_wait_ld<32>(v);
            if (!all) {
              hide(k, v);
              hide(k + 1, v + 16);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
              for (int c = 0; c < o; ++c) v[c] = fmaxf(v[c], v[c + o]);
            top = fmaxf(top, v[0]);
          };
#pragma unroll 1
          for (int k = 0; k < HC / 16; k += 2) top_of(k);
          if (!meet(top, theirs)) {
            gave_up();
            break;
          }
          const float up = fmaxf(m, fmaxf(top, theirs) * scl);
          // weights are relative to the maximum less kShift, which rounding must not take
          // far from it
          const float at = up == -INFINITY ? 0.f : up;
          float next = at - kShift;
          if (!(at - next <= kShift + 1.f)) next = at;
          alpha = m == -INFINITY ? 0.f : ex2(ref - next);
          m = up;
          ref = next;
          const u64 next2 = pair(-next, -next);
          const uint32_t third = lanes + C::kThird + buf * (TN / 2) + first / 2;
          u64 sum[2] = {0, 0};
          auto weights_of = [&](int k) {  // of 32 columns from 16 k on
            float v[32];
            tm_ld32(v, src + 16 * k);
            tm_wait_ld<32>(v);
            if (!all) {
              hide(k, v);
              hide(k + 1, v + 16);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t part[16], last[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                // rounded before the difference, as the maximum is (a packed product would be
                // fused with the sum: large scores' weights then lie anywhere)
                const float2 d = halves(add2(pair(__fmul_rn(v[16 * j + 2 * c], scl), __fmul_rn(v[16 * j + 2 * c + 1], scl)), next2));
                u64 p = pair(ex2(d.x), ex2(d.y));
                sum[c & 1] = add2(sum[c & 1], p);
                float2 f = halves(p);
                part[c] = round2<DT>(f.x, f.y);
                p = left2<DT>(p, part[c]);
                f = halves(p);
                part[8 + c] = round2<DT>(f.x, f.y);
                if constexpr (NP == 3) {
                  f = halves(left2<DT>(p, part[8 + c]));
                  last[c] = round2<DT>(f.x, f.y);
                }
              }
              tm_st16(src + 16 * (k + j), part);
              if constexpr (NP == 3) tm_st8(third + 8 * (k + j), last);
            }
          };
#pragma unroll 1
          for (int k = 0; k < HC / 16; k += 2) weights_of(k);
          const float2 both = halves(add2(sum[0], sum[1]));
          l = fmaf(l, alpha, both.x + both.y);
          tm_wait_st();
          tm_fence_before();
        }
        __syncwarp();
        if (lane == 0 && tile) mbar_arrive(&sh.pfull[buf]);
        if (i > walk.tile0) {
          const int ob = (t - 1) % NO;
          if (!wait_for(&sh.ofull[ob], (uint32_t)(((t - 1) / NO) & 1))) {
            gave_up();
            break;
          }
          if (live) {
            tm_fence_after();
            const u64 f2 = pair(before, before);
            float x[HO];
#pragma unroll
            for (int c0 = 0; c0 < HO; c0 += 32) tm_ld32(x + c0, lanes + C::kO + ob * DV + h * HO + c0);
            tm_wait_ld<HO>(x);
#pragma unroll
            for (int c = 0; c < HO / 2; ++c) o2[c] = fma2(o2[c], f2, pair(x[2 * c], x[2 * c + 1]));
            tm_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.oempty[ob]);
        }
        if (!tile) break;
      }
      if (!ok) break;
      const bool begins = walk.begins(), ends = walk.ends();
      if (begins && !ends && tid == 0)
        w.span[blockIdx.x] = TreeSpan{u.slot, u.unit, sh.line.block_of(sh.share0 + walk.at + tree_cost(MR, u.v.count) + u.tiles - 1), 1};
      const int dh = min(DV, D - u.half * 128) - h * HO;  // the half's columns of the unit's
      float o[HO];
      bool odd = false;
#pragma unroll
      for (int c = 0; c < HO / 2; ++c) {
        const float2 f = halves(o2[c]);
        o[2 * c] = f.x;
        o[2 * c + 1] = f.y;
      }
#pragma unroll
      for (int c = 0; c < HO; ++c) odd |= c < dh && !(fabsf(o[c]) < INFINITY);
      if (live) {
        float theirs = 0.f;
        if (odd) l = NAN;  // for the other half too
        if (!meet(l, theirs)) {
          gave_up();
          break;
        }
        l = h ? theirs + l : l + theirs;
      }
      if (!live) continue;
      const bool again = row < u.rows && !(l < INFINITY);
      const int R = u.row0 + row, draft = R / a.group;
      const size_t out = ((size_t)u.slot * a.drafts + draft) * a.heads + u.g * a.group + R - draft * a.group;
      float* part = w.part + ((size_t)(2 * blockIdx.x + begins) * MR + row) * (DV + 4);
      if (row < u.rows && !again) {
        if (begins && ends) {
          const float inv = l > 0.f ? 1.f / l : 0.f;
          float4* to = reinterpret_cast<float4*>(a.y + out * D + u.half * 128 + h * HO);
#pragma unroll
          for (int c = 0; c < HO; c += 4)
            if (c < dh) to[c / 4] = make_float4(o[c] * inv, o[c + 1] * inv, o[c + 2] * inv, o[c + 3] * inv);
          if (a.lse && u.half == 0 && h == 0) a.lse[out] = (ref + log2f(l)) * kLn2;
        } else {
#pragma unroll
          for (int c = 0; c < HO; c += 4)
            __stcg(reinterpret_cast<float4*>(part + h * HO + c), make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]));
          if (h == 0) __stcg(reinterpret_cast<float2*>(part + DV), make_float2(ref, l));
        }
      }
      for (uint32_t left = __ballot_sync(~0u, again); left; left &= left - 1) {
        const int r = (row & ~31) + __ffs(left) - 1;
        const RowSums s = tree_again<DT, TN, MR>(w, u, walk.tile0, walk.tile1, r, &sh.beat);
        const float inv = s.l > 0.f ? 1.f / s.l : s.l == s.l ? 0.f : s.l;
        const int Rr = u.row0 + r, dr = Rr / a.group, c = 8 * lane - 128 * u.half;
        const size_t to_row = ((size_t)u.slot * a.drafts + dr) * a.heads + u.g * a.group + Rr - dr * a.group;
        float* pr = w.part + ((size_t)(2 * blockIdx.x + begins) * MR + r) * (DV + 4);
        const bool direct = begins && ends;
        const float f = direct ? inv : 1.f;
        if (c >= h * HO && c < h * HO + HO && c < h * HO + dh) {
          float4* to = reinterpret_cast<float4*>(direct ? a.y + to_row * D + 8 * lane : pr + c);
          __stcg(to, make_float4(s.o[0] * f, s.o[1] * f, s.o[2] * f, s.o[3] * f));
          __stcg(to + 1, make_float4(s.o[4] * f, s.o[5] * f, s.o[6] * f, s.o[7] * f));
        }
        if (lane == 0 && h == 0) {
          if (!direct) __stcg(reinterpret_cast<float2*>(pr + DV), make_float2(s.m, s.l));
          else if (a.lse && u.half == 0) a.lse[to_row] = (s.m + log2f(s.l)) * kLn2;
        }
      }
    }
    } else {
    // ---- Q, softmax, O of few rows: a thread has a token of S and P, a column of V of O, in
    // both for half of the rows; Q lanes keep the figures of a row of the half
    constexpr int RH = MR / 2, Q = 32 / RH;
    const int h = warp >> 2, wq = warp & 3, place = 32 * wq + lane, own = lane / Q;
    const float flip = a.scale < 0.f ? -1.f : a.scale == 0.f ? 0.f : 1.f;
    const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale);
    constexpr float kShift = DT == 0 ? 14.f : 0.f;
    const uint32_t lanes = tmem + ((uint32_t)(32 * wq) << 16) + h * RH;
    int seg = 0, met = 0;
    // The four warps of a half show each other a value per row; false where the wait ran
    // out.
    auto meet = [&](float mine, float (&all)[4]) {
      if (lane % Q == 0) sh.few[met & 1][h][wq][own] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.pair[h]);
      if (!mbar_spin(&sh.pair[h], (uint32_t)(met & 1)) && !wait_for(&sh.pair[h], (uint32_t)(met & 1))) return false;
#pragma unroll
      for (int k = 0; k < 4; ++k) all[k] = sh.few[met & 1][h][k][own];
      ++met;
      return true;
    };
    for (; walk.more() && ok; walk.next()) {
      if (!walk.any()) continue;
      const TreeUnit& u = walk.u;
      // rows warp, warp + 8, ...: split into parts
      constexpr int E = DP / 32, B = MR / 8;
      float x[B][E];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int r = warp + 8 * b, R = u.row0 + r, i = R / a.group;
        const float* q = a.q + (((size_t)u.slot * a.drafts + i) * a.heads + u.g * a.group + R - i * a.group) * D + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e) x[b][e] = 0.f;
        if (r < u.rows && E * lane < D) {
          if constexpr (E == 2) {
            const float2 f = __ldg(reinterpret_cast<const float2*>(q));
            x[b][0] = f.x, x[b][1] = f.y;
          } else {
            const float4 f = __ldg(reinterpret_cast<const float4*>(q));
            x[b][0] = f.x, x[b][1] = f.y, x[b][E - 2] = f.z, x[b][E - 1] = f.w;
          }
        }
      }
      if (warp == 7) {  // what the rows see, a lane each
        int lo = 0;
        u64 seen = 0;
        if (lane < u.rows) {
          const int draft = (u.row0 + lane) / a.group;
          const u64 path = a.parent
              ? tree_path(a, draft, [&](int j) { return __ldg(a.parent + (size_t)u.slot * a.drafts + j); })
              : (2ull << draft) - 1;
          lo = a.window > 0 ? u.v.base + __popcll(path) - a.window : 0;
          seen = tree_seen(a, u.v.base, path);
        }
        sh.lo[seg & 1][lane] = lo;
        sh.seen[seg & 1][lane] = seen;
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int r = warp + 8 * b;
        float back = 1.f;
        if constexpr (DT == 0) {
          float top = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(x[b][e]));
          top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));
          const int ex = query_exponent(top);
          const float f = __uint_as_float((uint32_t)(ex + 127) << 23);
#pragma unroll
          for (int e = 0; e < E; ++e) x[b][e] *= f;
          back = __uint_as_float((uint32_t)(127 - ex) << 23);
        }
        if (lane == 0) sh.qs[seg & 1][r] = back;
        const int c = E * lane;
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = x[b][e] * flip;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          uint32_t part[E / 2];
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            part[e] = round2<DT>(y[2 * e], y[2 * e + 1]);
            y[2 * e] -= from_bits<DT>((uint16_t)part[e]);
            y[2 * e + 1] -= from_bits<DT>((uint16_t)(part[e] >> 16));
          }
          const int n = p * MR + r;
          unsigned char* to = smem + (c >> 6) * kPanelQ + n * 128 + ((((c >> 3) & 7) ^ (n & 7)) << 4) + 2 * (c & 7);
          if constexpr (E == 2) *reinterpret_cast<uint32_t*>(to) = part[0];
          else *reinterpret_cast<uint2*>(to) = make_uint2(part[0], part[E / 2 - 1]);
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.qfull);
      TREE_WAIT(&sh.qfull, seg & 1);
      const bool live = h * RH < u.rows;
      const float scl = scale * sh.qs[seg & 1][h * RH + own];
      const int* const los = sh.lo[seg & 1] + h * RH;
      const u64* const seens = sh.seen[seg & 1] + h * RH;
      const int sinks = u.v.tail > 0 ? 0 : a.sinks;
      float m = -INFINITY, ref = -INFINITY, alpha = 0.f;
      float l[RH], o[RH];
#pragma unroll
      for (int j = 0; j < RH; ++j) l[j] = o[j] = 0.f;
      // the sum of a row's parts, lowest first
      auto load = [&](float (&v)[RH], uint32_t from) {
        float z[NP][RH];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          if constexpr (RH == 16) tm_ld16(z[p], from + p * MR);
          else tm_ld8(z[p], from + p * MR);
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) tm_wait_ld<RH>(z[p]);
#pragma unroll
        for (int j = 0; j < RH; ++j) v[j] = NP == 3 ? (z[NP - 1][j] + z[1][j]) + z[0][j] : z[1][j] + z[0][j];
      };
      for (int i = walk.tile0;; ++i, ++t) {  // the softmax of tile i, then the sums with tile i - 1's O
        const int buf = t & 1;
        const float before = alpha;
        const bool tile = i < walk.tile1;
        if (tile) TREE_WAIT(&sh.sfull[buf], (t >> 1) & 1);
        if (live && tile) {
          tm_fence_after();
          float v[RH];
          load(v, lanes + buf * NQ);
          int any_lo = 0, hi = 0, t0 = 0;
          if (i > 0) t0 = walk.cached(i, any_lo, hi);
          const int tok = t0 + place;
          const bool past = place >= hi - t0;
          const bool gone = sh.hide[t % kTreeHide][wq] >> lane & 1u;
          // a window's tokens from base + 1 on below the deepest row's are not seen by all
          if (i == 0) {
#pragma unroll
            for (int j = 0; j < RH; ++j)
              v[j] = place < 64 && (seens[j] >> (place & 63) & 1) && !gone ? v[j] : -INFINITY;
          } else if (i <= u.firsts || a.window == 0) {
            if (__any_sync(~0u, past || gone)) {
#pragma unroll
              for (int j = 0; j < RH; ++j) v[j] = !past && !gone ? v[j] : -INFINITY;
            }
          } else if (__any_sync(~0u, past || gone || tok - PI_TREE_MAX < u.v.base - a.window)) {
#pragma unroll
            for (int j = 0; j < RH; ++j)
              v[j] = !past && !gone && (tok >= los[j] || tok < sinks) ? v[j] : -INFINITY;
          }
          float tops[4];
          float most[RH];
#pragma unroll
          for (int j = 0; j < RH; ++j) most[j] = v[j];
          if (!meet(warp_rows(most, [](float x, float y) { return fmaxf(x, y); }), tops)) {
            gave_up();
            break;
          }
          const float up = fmaxf(m, fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scl);
          const float at = up == -INFINITY ? 0.f : up;
          float next = at - kShift;
          if (!(at - next <= kShift + 1.f)) next = at;
          alpha = m == -INFINITY ? 0.f : ex2(ref - next);
          m = up;
          ref = next;
          unsigned char* const pt = smem + C::kWeights + buf * C::kP + place * 128;
          u64 p[RH / 2];
          __syncwarp();
          if (lane % Q == 0) sh.figures[warp][own] = make_float4(scl, next, alpha, before);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < RH; ++j) {
            const float4 f = sh.figures[warp][j];
            v[j] = ex2(__fmul_rn(v[j], f.x) - f.y);
            l[j] = fmaf(l[j], f.z, v[j]);
          }
#pragma unroll
          for (int j = 0; j < RH / 2; ++j) p[j] = pair(v[2 * j], v[2 * j + 1]);
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            uint32_t part[RH / 2];
#pragma unroll
            for (int j = 0; j < RH / 2; ++j) {
              const float2 f = halves(p[j]);
              part[j] = round2<DT>(f.x, f.y);
              if (k + 1 < NP) p[j] = left2<DT>(p[j], part[j]);
            }
            const int n = k * MR + h * RH;
#pragma unroll
            for (int j = 0; j < RH / 8; ++j)
              *reinterpret_cast<uint4*>(pt + ((n + 8 * j) >> 6) * kPanelK + (((((n + 8 * j) >> 3) & 7) ^ (place & 7)) << 4)) =
                  make_uint4(part[4 * j], part[4 * j + 1], part[4 * j + 2], part[4 * j + 3]);
          }
          fence_async();
          tm_fence_before();
        }
        __syncwarp();
        if (lane == 0 && tile) mbar_arrive(&sh.pfull[buf]);
        if (i > walk.tile0) {
          const int ob = (t - 1) % NO;
          if (!wait_for(&sh.ofull[ob], (uint32_t)(((t - 1) / NO) & 1))) {
            gave_up();
            break;
          }
          if (live) {
            tm_fence_after();
            float x[RH];
            load(x, lanes + C::kO + ob * NQ);
#pragma unroll
            for (int j = 0; j < RH; ++j) {
              const float4 f = sh.figures[warp][j];
              o[j] = fmaf(o[j], tile ? f.w : f.z, x[j]);
            }
            tm_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.oempty[ob]);
        }
        if (!tile) break;
      }
      if (!ok) break;
      ++seg;
      const bool begins = walk.begins(), ends = walk.ends(), direct = begins && ends;
      if (begins && !ends && tid == 0)
        w.span[blockIdx.x] = TreeSpan{u.slot, u.unit, sh.line.block_of(sh.share0 + walk.at + tree_cost(MR, u.v.count) + u.tiles - 1), 1};
      if (!live) continue;
      const int dh = min(DV, D);
#pragma unroll
      for (int j = 0; j < RH; ++j)
        if (place < dh && !(fabsf(o[j]) < INFINITY)) l[j] = NAN;
      float sums[4];
      if (!meet(warp_rows(l, [](float x, float y) { return x + y; }), sums)) {
        gave_up();
        break;
      }
      const float sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
      const int r = h * RH + own, R = u.row0 + r, draft = R / a.group;
      const int out = (u.slot * a.drafts + draft) * a.heads + u.g * a.group + R - draft * a.group;
      const bool good = r < u.rows && sum < INFINITY, again = r < u.rows && !good;
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const uint32_t rows = __ballot_sync(~0u, good);
      float* const part = w.part + ((size_t)(2 * blockIdx.x + begins) * MR + h * RH) * (DV + 4);
      if (wq == 0 && lane % Q == 0 && good) {
        if (!direct) __stcg(reinterpret_cast<float2*>(part + own * (DV + 4) + DV), make_float2(ref, sum));
        else if (a.lse) a.lse[out] = (ref + log2f(sum)) * kLn2;
      }
#pragma unroll
      for (int j = 0; j < RH; ++j) {
        const float f = __shfl_sync(~0u, inv, j * Q);
        const int to = __shfl_sync(~0u, out, j * Q);
        if (place < dh && rows >> (j * Q) & 1u) {
          if (direct) a.y[(size_t)to * D + place] = o[j] * f;
          else __stcg(part + j * (DV + 4) + place, o[j]);
        }
      }
      // a row in four to each of the half's warps
      for (uint32_t left = __ballot_sync(~0u, again && lane % Q == 0 && (own & 3) == wq); left; left &= left - 1) {
        const int j = (__ffs(left) - 1) / Q;
        const RowSums s = tree_again<DT, TN, MR>(w, u, walk.tile0, walk.tile1, h * RH + j, &sh.beat);
        const float f = !direct ? 1.f : s.l > 0.f ? 1.f / s.l : s.l == s.l ? 0.f : s.l;
        const int to_row = __shfl_sync(~0u, out, j * Q);
        float* pr = part + j * (DV + 4);
        if (8 * lane < dh) {
          float4* to = reinterpret_cast<float4*>(direct ? a.y + (size_t)to_row * D + 8 * lane : pr + 8 * lane);
          __stcg(to, make_float4(s.o[0] * f, s.o[1] * f, s.o[2] * f, s.o[3] * f));
          __stcg(to + 1, make_float4(s.o[4] * f, s.o[5] * f, s.o[6] * f, s.o[7] * f));
        }
        if (lane == 0) {
          if (!direct) __stcg(reinterpret_cast<float2*>(pr + DV), make_float2(s.m, s.l));
          else if (a.lse) a.lse[to_row] = (s.m + log2f(s.l)) * kLn2;
        }
      }
    }
    }
  } else if (warp == 8) {
    // ---- MMAs
    int seg = 0, cols_before = 0, nv_before = 0;
    auto pv = [&](int p, int cols, int nv) {  // tile p's O
      const int buf = p & 1, st = p % SV, ob = p % NO;
      if (!wait_for(&sh.vfull[st], (uint32_t)((p / SV) & 1)) ||
          !wait_for(&sh.pfull[buf], (uint32_t)((p >> 1) & 1)) ||
          (p >= NO && !wait_for(&sh.oempty[ob], (uint32_t)(((p / NO) - 1) & 1)))) {
        gave_up();
        return;
      }
      tm_fence_after();
      if (elected()) {
        const uint32_t d = tmem + C::kO + ob * C::kO1;
        const uint32_t vs = smem_u32(smem + C::kValues + st * C::kV);
        if constexpr (kFew) {  // V^T (rows from DV on are not looked at) by P
          const uint64_t vd = tree_desc(vs, DV == 128 ? kPanelK : 0);
          const uint64_t pd = tree_desc(smem_u32(smem + C::kWeights + buf * C::kP), kPanelK);
          const uint32_t idesc = tree_idesc<DT>(NQ, true, true);
#pragma unroll
          for (int ks = 0; ks < TN / 16; ++ks)
            if (16 * ks < cols) mma_ss(d, vd + (2048 >> 4) * ks, pd + (2048 >> 4) * ks, idesc, ks > 0);
        } else {
          const uint64_t vd = tree_desc(vs, kPanelK);
          const uint32_t idesc = tree_idesc<DT>(nv, true);
          bool add = false;
#pragma unroll
          for (int part = NP - 1; part >= 0; --part) {
            const uint32_t pa = part == 2 ? tmem + C::kThird + buf * (TN / 2) : tmem + buf * TN + part * 8;
#pragma unroll
            for (int ks = 0; ks < TN / 16; ++ks)
              if (16 * ks < cols) {
                mma_ts(d, pa + (part == 2 ? 8 : 16) * ks, vd + (2048 >> 4) * ks, idesc, add);
                add = true;
              }
          }
        }
        mma_commit(&sh.vempty[st]);
        mma_commit(&sh.ofull[ob]);
      }
      __syncwarp();
    };
    for (; walk.more() && ok; walk.next()) {
      if (!walk.any()) continue;
      const int nv = (min(DV, D - walk.u.half * 128) + 15) & ~15;
      for (int i = walk.tile0; i < walk.tile1 && ok; ++i, ++t) {
        const int st = t % SK, buf = t & 1, cols = walk.columns(i);
        if (i == walk.tile0) {
          if (t > 0) pv(t - 1, cols_before, nv_before);
          if (!ok) break;
          TREE_WAIT(&sh.qfull, seg & 1);
        }
        TREE_WAIT(&sh.kfull[st], (t / SK) & 1);
        tm_fence_after();
        if (elected()) {
          const uint64_t qd = tree_desc(smem_u32(smem), 16);
          const uint64_t kdesc = tree_desc(smem_u32(smem + C::kStages + st * C::kK), 16);
          if constexpr (kFew) {  // K by Q^T
            const uint32_t idesc = tree_idesc<DT>(NQ, false);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
              if (k < kd)
                mma_ss(tmem + buf * NQ, kdesc + (((k >> 2) * kPanelK + (k & 3) * 32) >> 4),
                       qd + (((k >> 2) * kPanelQ + (k & 3) * 32) >> 4), idesc, k > 0);
          } else {
            const uint32_t idesc = tree_idesc<DT>(cols, false);
            bool add = false;
#pragma unroll
            for (int part = NP - 1; part >= 0; --part)
#pragma unroll
              for (int k = 0; k < DP / 16; ++k)
                if (k < kd) {
                  mma_ss(tmem + buf * TN, qd + ((part * C::kQ + (k >> 2) * kPanelQ + (k & 3) * 32) >> 4),
                         kdesc + (((k >> 2) * kPanelK + (k & 3) * 32) >> 4), idesc, add);
                  add = true;
                }
          }
          mma_commit(&sh.kempty[st]);
          mma_commit(&sh.sfull[buf]);
        }
        __syncwarp();
        if (i > walk.tile0) pv(t - 1, cols_before, nv_before);
        cols_before = cols;
        nv_before = nv;
      }
      ++seg;
    }
    if (ok && t > 0) pv(t - 1, cols_before, nv_before);
  } else {
    // ---- K, or V
    const bool value = warp >= 9 + C::KW;
    const int pw = warp - 9 - (value ? C::KW : 0), warps = value ? C::VW : C::KW;  // of the operand's warps
    const int stages = value ? SV : SK;
    uint64_t* const full = value ? sh.vfull : sh.kfull;
    uint64_t* const empty = value ? sh.vempty : sh.kempty;
    const size_t half = (size_t)a.kv_heads * P * D;  // K to V in a page
    // self-test: a copy that nobody orders, of the first keys before slot 0's drafts; the
    // unit is its block's first (a condition within the loop costs 2 % of the
    // largest case)
    if (w.lose && !value && pw == 0 && lane == 0 && walk.more() && (walk.u.slot | walk.u.unit) == 0 &&
        walk.tile0 <= 1 && walk.tile1 > 1)
      mbar_expect_more(full + 1 - walk.tile0, 128);
    for (; walk.more() && ok; walk.next()) {
      if (!walk.any()) continue;
      const TreeUnit& u = walk.u;
      const int dh = min(DV, D - u.half * 128);                  // the unit's columns of V
      const int d0 = value ? u.half * 128 : 0, d1 = value ? dh : D;  // the operand's elements of a row
      const int panels = (d1 + 63) >> 6, pieces = value ? ((dh + 15) & ~15) >> 3 : 2 * kd;  // of 16 bytes
      auto index_of = [&](int tok) { return w.page_shift >= 0 ? tok >> w.page_shift : tok / P; };
      auto row_of = [&](int tok) -> const uint16_t* {  // null: page out of range
        const int j = index_of(tok);
        const int page = checked_page(__ldg(a.table + (size_t)u.slot * a.max_pages + j), a.pages, a.status);
        return page < 0 ? nullptr
                        : a.pool + (((size_t)page * 2 * a.kv_heads + u.g) * P + tok - j * P) * D + (value ? half : 0) + d0;
      };
      // Lane b's box of a tile: whether it is seen, its page and its row of the pool; read
      // a tile ahead.
      struct Boxes {
        int t0, lo, hi, box, page, row;
        bool whole, some;
      };
      auto boxes_of = [&](int i) {
        Boxes x{u.v.base, u.v.base, u.v.base + u.v.count, 0, 0, 0, false, false};  // the drafts
        if (i == 0 || i >= walk.tile1) return x;
        x.t0 = walk.cached(i, x.lo, x.hi);
        if (!w.tma) return x;
        x.whole = x.t0 >= x.lo && x.hi - x.t0 >= TN;
        x.box = x.whole ? w.box : w.edge;
        const int at = lane * x.box;
        x.some = at < TN && at + x.box > x.lo - x.t0 && at < x.hi - x.t0;
        if (x.some) {
          const int b0 = x.t0 + at, j = index_of(b0);
          x.page = __ldg(a.table + (size_t)u.slot * a.max_pages + j);
          x.row = b0 - j * P;
        }
        return x;
      };
      // the rows of q are read when the warps 0-7 come to the segment
      if (value)
        for (int e = 32 * pw + lane; e < u.rows * ((D + 31) / 32); e += 32 * C::VW) {
          const int r = e / ((D + 31) / 32), R = u.row0 + r, d = R / a.group;
          const float* q = a.q + (((size_t)u.slot * a.drafts + d) * a.heads + u.g * a.group + R - d * a.group) * D +
                           32 * (e - r * ((D + 31) / 32));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
        }
      const int be = pw + warps * lane;  // the lane's box and panel of a tile
      const int bb = panels == 1 ? be : panels == 2 ? be >> 1 : panels == 4 ? be >> 2 : be / panels, bp = be - bb * panels;
      Boxes ahead = boxes_of(walk.tile0);
      for (int i = walk.tile0; i < walk.tile1; ++i, ++t) {
        const int round = t / stages, st = t - round * stages;
        unsigned char* const to = smem + (value ? C::kValues + st * C::kV : C::kStages + st * C::kK);
        const Boxes now = ahead;
        const int t0 = now.t0, lo = now.lo, hi = now.hi;
        const int cols = i == 0 ? (u.v.count + 15) & ~15 : (min(TN, hi - t0) + 15) & ~15;
        const bool boxes = now.box && __all_sync(~0u, !now.some || (unsigned)now.page < (unsigned)a.pages);
        const bool fresh = i == 0 && a.k_new;
        ahead = boxes_of(i + 1);
        const int box_row = __shfl_sync(~0u, (now.page * 2 * a.kv_heads + u.g) * P + now.row, bb & 31) +
                            (value ? a.kv_heads * P : 0);
        if (round > 0) TREE_WAIT(empty + st, (round - 1) & 1);
        if (!value && pw == 0) {
          if (boxes || fresh) {
            if (lane < TN / 32) sh.hide[t % kTreeHide][lane] = 0;
          } else {
#pragma unroll 1
            for (int k = 0; k < TN / 32; ++k) {
              const int tok = t0 + 32 * k + lane;
              const uint32_t h = __ballot_sync(~0u, tok >= lo && 32 * k + lane < hi - t0 && !row_of(tok));
              if (lane == 0) sh.hide[t % kTreeHide][k] = h;
            }
          }
        }
        // Rows by hand, zeros where nobody sees a row or its page is out of range: all
        // of them, or those of V in boxes that are not seen whole.  New drafts are
        // rounded to the cache's type, and stored by the first unit of their kv head.
        if (!boxes || (value && !now.whole)) {
          auto piece = [&](int r, int e) {
            const int tok = t0 + r;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (tok < lo || r >= hi - t0 || e >= d1) return x;
            if (!fresh) {
              const uint16_t* row = row_of(tok);
              return row ? *reinterpret_cast<const uint4*>(row + e) : x;
            }
            const float4* f = reinterpret_cast<const float4*>(
                (value ? a.v_new : a.k_new) + (((size_t)u.slot * a.drafts + r) * a.kv_heads + u.g) * D + d0 + e);
            const float4 y = __ldg(f), z = __ldg(f + 1);
            return make_uint4(round2<DT>(y.x, y.y), round2<DT>(y.z, y.w), round2<DT>(z.x, z.y), round2<DT>(z.z, z.w));
          };
          const bool keep = fresh && u.row0 == 0 && (value || u.half == 0);
#pragma unroll 1
          for (int r0 = 0; r0 < cols;) {
            const int rows = boxes ? now.box : cols, n = rows * pieces;
            if (!boxes || r0 < lo - t0 || r0 + rows > hi - t0) {
#pragma unroll 1
              for (int e0 = 32 * pw + lane; e0 < n; e0 += 128 * warps) {
                uint4 x[4];
                int r[4], c[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int e = min(e0 + 32 * warps * k, n - 1);
                  r[k] = e / pieces;
                  c[k] = e - r[k] * pieces;
                  r[k] += r0;
                  x[k] = piece(r[k], 8 * c[k]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  *reinterpret_cast<uint4*>(to + (c[k] >> 3) * kPanelK + r[k] * 128 + (((c[k] & 7) ^ (r[k] & 7)) << 4)) = x[k];
                  if (keep && r[k] < hi - t0 && 8 * c[k] < d1)
                    if (const uint16_t* row = row_of(t0 + r[k]))
                      *reinterpret_cast<uint4*>(const_cast<uint16_t*>(row) + 8 * c[k]) = x[k];
                }
              }
            }
            r0 += rows;
          }
          fence_async();
        }
        __syncwarp();
        // TMA: a box of K where anything of it is seen, of V where all of it is
        const int r = bb * now.box;  // of the tile
        const bool mine = boxes && r < cols && (now.whole || (value ? r >= lo - t0 && r + now.box <= hi - t0
                                                                    : r + now.box > lo - t0 && r < hi - t0));
        const int n = __popc(__ballot_sync(~0u, mine));
        if (lane == 0) mbar_expect(full + st, (uint32_t)(n * now.box * 128));
        __syncwarp();
        if (mine)
          tree_box(smem_u32(to + bp * kPanelK + r * 128), now.whole ? &map : &edge_map, d0 + 64 * bp, box_row, full + st);
      }
    }
  }
#undef TREE_WAIT
  tm_fence_before();
  __syncthreads();
  if (sh.bad) {  // copies and MMAs under way come to their end (2 s at most)
    if (warp >= 9) {
      const bool value = warp >= 9 + C::KW;
      const int stages = value ? SV : SK;
      for (int i = 0; i < stages && i < t; ++i)
        mbar_wait((value ? sh.vfull : sh.kfull) + i, (uint32_t)((t - 1 - i) / stages & 1), 500000000ull);
    }
    if (warp == 8) {
      if (elected()) mma_commit(&sh.fin);  // it covers the MMAs of the lane that issued them
      __syncwarp();
      mbar_wait(&sh.fin, 0, 2000000000ull);
    }
    __syncthreads();
  }
  if (warp == 8) {
    tm_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Joins the parts of the units that several blocks share: a warp per row.
template <int DT, int DP, int MR>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ TreeWork w) {
  using C = TreeTile<DT, DP, MR>;
  constexpr int DV = C::DV;
  pdl_enter();
  const TreeArgs& a = w.a;
  const TreeSpan sp = w.span[blockIdx.x];
  if (!sp.some) return;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  TreeWalk<C::TN, MR> walk(w, sp.slot, sp.unit, 0, 1, true);
  const TreeUnit& u = walk.u;
  if (r >= u.rows) return;
  const int n = sp.last - blockIdx.x + 1, dh = min(DV, a.head_dim - u.half * 128);
  float top = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const float* pr = w.part + ((size_t)(2 * (blockIdx.x + j) + (j == 0)) * MR + r) * (DV + 4);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(pr + DV));
    const float4 x = 4 * lane < DV ? __ldcg(reinterpret_cast<const float4*>(pr + 4 * lane)) : o;
    // a part of nothing that is seen has the sum 0
    const float up = ml.y == 0.f ? top : fmaxf(top, ml.x), ref = up == -INFINITY ? 0.f : up;
    const float was = part_weight(top - ref), is = ml.y == 0.f ? 0.f : part_weight(ml.x - ref);
    o.x = fmaf(x.x, is, o.x * was);
    o.y = fmaf(x.y, is, o.y * was);
    o.z = fmaf(x.z, is, o.z * was);
    o.w = fmaf(x.w, is, o.w * was);
    l = fmaf(ml.y, is, l * was);
    top = up;
  }
  const int R = u.row0 + r, draft = R / a.group;
  const size_t out = ((size_t)u.slot * a.drafts + draft) * a.heads + u.g * a.group + R - draft * a.group;
  const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
  if (4 * lane < dh)
    *reinterpret_cast<float4*>(a.y + out * a.head_dim + u.half * 128 + 4 * lane) =
        make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (lane == 0 && a.lse && u.half == 0) a.lse[out] = (top + log2f(l)) * kLn2;
}

template <int DT, int DP, int MR>
static pi_status launch_tree(TreeWork& w, const CUtensorMap& map, const CUtensorMap& edge_map, const DevInfo& di,
                             pi_stream stream) {
  using C = TreeTile<DT, DP, MR>;
  constexpr int smem = tree_smem<DT, DP, MR>();
  static_assert(smem <= 232448, "shared memory");
  pi_status st = ensure_smem(reinterpret_cast<const void*>(tree_kernel<DT, DP, MR>), smem);
  if (st != PI_OK) return st;
  // all blocks that are resident together, or fewer where the longest slots that the
  // tables and the window allow cannot use them
  const TreeArgs& a = w.a;
  long long seen = (long long)a.max_pages * a.page_tokens;
  if (a.window > 0 && (long long)a.window + a.sinks < seen) seen = (long long)a.window + a.sinks;
  const long long units = (long long)a.slots * a.kv_heads * ((a.drafts * a.group + MR - 1) / MR) * w.halves;
  const long long most = (seen + 63) / C::TN + 4;  // tiles of a unit
  const bool whole = most <= kTreeWhole;
  const long long useful = whole ? units : units * (most + tree_cost(MR, a.drafts));
  long long grid = di.sms < kTreeGrid ? di.sms : kTreeGrid;
  if (grid > useful) grid = useful;
  st = launch(tree_kernel<DT, DP, MR>, dim3((unsigned)grid), C::kThreads, smem, stream, w, map,
              edge_map);
  if (st != PI_OK || whole || grid < 2) return st;
  const int rows = a.drafts * a.group < MR ? a.drafts * a.group : MR;
  return launch(tree_join_kernel<DT, DP, MR>, dim3((unsigned)(grid - 1), (unsigned)((rows + 7) / 8)), 256, 0, stream, w);
}

template <int DT>
static pi_status launch_rows(TreeWork& w, const CUtensorMap& map, const CUtensorMap& edge_map, const DevInfo& di,
                             pi_stream stream) {
  const int rows = w.a.drafts * w.a.group;
  if (w.a.head_dim <= 64)
    return rows <= 16   ? launch_tree<DT, 64, 16>(w, map, edge_map, di, stream)
           : rows <= 32 ? launch_tree<DT, 64, 32>(w, map, edge_map, di, stream)
                        : launch_tree<DT, 64, 128>(w, map, edge_map, di, stream);
  if (w.a.head_dim <= 128)
    return rows <= 16   ? launch_tree<DT, 128, 16>(w, map, edge_map, di, stream)
           : rows <= 32 ? launch_tree<DT, 128, 32>(w, map, edge_map, di, stream)
                        : launch_tree<DT, 128, 128>(w, map, edge_map, di, stream);
  return launch_tree<DT, 256, 64>(w, map, edge_map, di, stream);
}

// Map over a layer's rows (K and V rows of every page and kv head): boxes of 64
// elements of `box` rows, 128-byte swizzle, zeros past a row's end.
static bool tree_map(CUtensorMap* m, void* base, long long rows, int head_dim, int box) {
  const EncodeFn encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)head_dim, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)head_dim * 2};
  const cuuint32_t boxes[2] = {64u, (cuuint32_t)box}, steps[2] = {1u, 1u};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, dims, strides, boxes, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The spans' place in a workspace, and the parts' behind them.
constexpr size_t kTreeSpans = kCounters;
constexpr size_t kTreeParts = kTreeSpans + (kTreeGrid * sizeof(TreeSpan) + kAlign - 1) / kAlign * kAlign;

}  // namespace pis

using namespace pis;

extern "C" {

size_t pi_tree_workspace_size(const pi_cache_desc* cache, int32_t slots, int32_t heads, int32_t drafts) {
  if (check_cache(cache) != PI_OK || slots < 1 || slots > PI_CACHE_MAX_SLOTS) return 0;
  if (heads < 1 || heads > kMaxHeads || heads % cache->kv_heads || drafts < 1 || drafts > PI_TREE_MAX) return 0;
  const int dv = cache->head_dim <= 64 ? 64 : 128;
  return kTreeParts + (size_t)kTreeGrid * 2 * (cache->head_dim > 128 ? 64 : 128) * (dv + 4) * 4;
}

}  // extern "C"

static pi_status tree_attention(const pi_cache_desc* cache, int32_t layer, int32_t slots, int32_t heads,
                                int32_t max_pages, int32_t drafts, const int32_t* parent, const int32_t* count,
                                const float* q, const float* k_new, const float* v_new, const int32_t* table,
                                const int32_t* len, void* pool, float scale, int32_t window, int32_t sinks,
                                float* y, float* lse, int32_t* dev_status, void* ws, size_t ws_bytes,
                                pi_stream stream, unsigned long long lose_ns) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  const pi_cache_desc& C = *cache;
  st = check_slots(C, slots, max_pages);
  if (st != PI_OK) return st;
  if (layer < 0 || layer >= C.layers || heads < 1 || heads > kMaxHeads || heads % C.kv_heads) return PI_ERR_SHAPE;
  if (drafts < 1 || drafts > PI_TREE_MAX || window < 0 || sinks < 0) return PI_ERR_SHAPE;
  if (!q || !table || !len || !pool || !y || !dev_status || !ws || !k_new != !v_new) return PI_ERR_NULL;
  if (!all_aligned(parent, count, q, k_new, v_new, table, len, pool, y, lse, dev_status, ws)) return PI_ERR_ALIGN;
  if (ws_bytes < pi_tree_workspace_size(cache, slots, heads, drafts)) return PI_ERR_WORKSPACE;
  if (y == q) return PI_ERR_SHAPE;  // blocks that share rows read q while others write y
  TreeArgs a{};
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.parent = parent;
  a.count = count;
  a.table = table;
  a.len = len;
  a.pool = static_cast<uint16_t*>(pool) + (size_t)layer * C.pages * page_elems(C);
  a.y = y;
  a.lse = lse;
  a.status = dev_status;
  a.slots = slots;
  a.drafts = drafts;
  a.heads = heads;
  a.kv_heads = C.kv_heads;
  a.group = heads / C.kv_heads;
  a.head_dim = C.head_dim;
  a.page_tokens = C.page_tokens;
  a.pages = C.pages;
  a.max_pages = max_pages;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale * 1.4426950408889634f;
  TreeWork w{};
  w.a = a;
  w.span = reinterpret_cast<TreeSpan*>(static_cast<char*>(ws) + kTreeSpans);
  w.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kTreeParts);
  w.halves = C.head_dim > 128 ? 2 : 1;
  w.limit_ns = lose_ns ? lose_ns : wait_limit();
  w.lose = lose_ns != 0;
  const long long rows = (long long)C.pages * 2 * C.kv_heads * C.page_tokens;
  CUtensorMap map = {}, edge_map = {};
  w.box = C.page_tokens & -C.page_tokens;
  w.box = w.box < 64 ? w.box : 64;
  w.edge = w.box < 16 ? w.box : 16;
  w.align = w.box > 16 ? w.box : 16;
  w.page_shift = C.page_tokens & (C.page_tokens - 1) ? -1 : __builtin_ctz((unsigned)C.page_tokens);
  w.tma = w.box >= 8 && C.head_dim >= 64 && rows < (1ll << 31) &&
          tree_map(&map, a.pool, rows, C.head_dim, w.box) &&
          tree_map(&edge_map, a.pool, rows, C.head_dim, w.edge);
  if (lose_ns && !w.tma) return PI_ERR_SHAPE;
  DevInfo di;
  st = dev_info(&di);
  if (st != PI_OK) return st;
  const bool f16 = C.dtype == PI_F16;
  return f16 ? launch_rows<0>(w, map, edge_map, di, stream) : launch_rows<1>(w, map, edge_map, di, stream);
}

extern "C" {

pi_status pi_tree_attention(const pi_cache_desc* cache, int32_t layer, int32_t slots, int32_t heads,
                            int32_t max_pages, int32_t drafts, const int32_t* parent, const int32_t* count,
                            const float* q, const float* k_new, const float* v_new, const int32_t* table,
                            const int32_t* len, void* pool, float scale, int32_t window, int32_t sinks,
                            float* y, float* lse, int32_t* dev_status, void* ws, size_t ws_bytes,
                            pi_stream stream) {
  return tree_attention(cache, layer, slots, heads, max_pages, drafts, parent, count, q, k_new, v_new, table, len,
                        pool, scale, window, sinks, y, lse, dev_status, ws, ws_bytes, stream, 0);
}

pi_status pi_selftest_tree_timeout(const pi_cache_desc* cache, int32_t slots, int32_t heads, int32_t max_pages,
                                   int32_t drafts, const float* q, const int32_t* table, const int32_t* len,
                                   void* pool, float* y, int32_t* dev_status, void* ws, size_t ws_bytes,
                                   int64_t limit_ns, pi_stream stream) {
  if (limit_ns < 1000 || limit_ns > 5000000000LL) return PI_ERR_SHAPE;
  return tree_attention(cache, 0, slots, heads, max_pages, drafts, nullptr, nullptr, q, nullptr, nullptr, table, len,
                        pool, 1.f, 0, 0, y, nullptr, dev_status, ws, ws_bytes, stream, (unsigned long long)limit_ns);
}

}  // extern "C"
