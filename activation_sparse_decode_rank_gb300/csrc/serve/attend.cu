// attend.cu — attention of one new token per slot over a paged cache, and
// the stores of new keys and values (include/pi_serve.h).
#include <cuda.h>

#include <cstdlib>

#include "serve.cuh"

namespace pis {

// ------------------------------------------------------------------ attention
//
// Mathematics.  A query head's visible tokens may be split into any parts;
// part i yields m_i = max a_t, l_i = sum exp(a_t - m_i), o_i = sum exp(a_t -
// m_i) v_t, and parts join with the weights exp(m_i - max m).  Everything
// below is that, at three levels: tiles of 16 tokens within a warp, the four
// warps of a block, the blocks that share one (slot, kv head).
//
// Bound: each cache row is read once, so HBM bandwidth; with 8 query heads
// per kv head there are 16 multiply-adds per byte, too many for the FP32
// pipes beside the conversions, so both products run on the tensor cores.
//
// Tensor-core form (mma m16n8k16).  Rows 0..7 of the 16-row operand hold
// eight query heads' high 16-bit parts, rows 8..15 their low parts: one
// instruction multiplies both, the sum of accumulator rows h and h + 8 is
// the 22-bit product, and each lane finds both in its own registers.  The
// weights p = exp2(.) of the second product are split the same way.  bf16
// parts hold 8 bits each, so that type takes a second instruction with the
// third part (q's in halves, so that no row of it is 0).  fp16's narrow
// exponent range is met by exact powers of two: q is scaled to [2^13, 2^14) per
// head, and p's reference is the maximum less 14, so that the largest p is 2^14.
//
// Work split.  The tiles of all (slot, kv head, head tile) units, each unit
// preceded by kUnitCost positions that stand for its fixed cost, form one
// line; each warp takes an equal contiguous share of it, found from the
// lengths on the device, so ragged lengths balance and nothing depends on the
// host knowing them.  Short units have a block or a warp each (kApartTiles,
// kWholeTiles).  A unit inside one warp's share is written from that
// warp's registers.  A unit that spans warps leaves partial results, joined
// once at the end: within a thread block through shared memory, across
// thread blocks by the last of them to arrive, in block order, in groups first
// where they are many (no waiting; the order of the sums is fixed).
//
// Data flow.  A warp streams its tiles through its own ring of stages, without
// any block-wide barrier until the end.  Where pages hold multiples of 16 (8)
// tokens, a tile (half a tile) lies in one page: one lane orders its K and V
// as TMA boxes of 16 (8) rows, 128-byte swizzle, that arrive on the stage's
// mbarrier (values of rows outside the visible set are cleared before use).
// Other page sizes, head dimensions below 64 and pools of 2^31 rows or more
// gather row pieces with cp.async into the same layout.  Head dimensions below
// 64, 128 or 256 are padded with zeros in shared memory only.
//
// Measured, bytes of the rows seen against a copy's 6.8 TB/s.  32 slots x 40
// heads of 128, lengths to 2048, fp16: 109 us, 91 %.  8 slots, 64/8 heads of
// 128, lengths to 131072, bf16: 302 us, 97 %.  24 slots, 32/8 heads of 128, a
// window of 1000: 28.4 us, 49 %, of which 5 to the first tile and 5 in joins.
// One slot, 16 heads of 64, 200 tokens: 8.3 us, all latency; an empty launch in
// its place takes 0.8, one that ends after finding its share 3.
struct AttendArgs {
  const float *q, *k_new, *v_new;
  const int *table, *len;
  uint16_t* pool;  // the layer's pages
  float *y, *lse;
  int* status;
  int* arrived;   // [2][kAttendGrid] arrivals at the units that begin in a block, at groups
  float* part;    // [grid][2][heads of a unit][head_dim + 4]: o, m, l of units split over blocks
  int slots, heads, kv_heads, group, head_dim, page_tokens, pages, max_pages, window, sinks;
  int tiles;      // head tiles per kv head: ceil(group / 8)
  int page_shift; // log2(page_tokens), or -1
  int tma;        // tiles come as TMA boxes: 1 of a panel, 2 of all panels
  float scale;    // scale log2(e)
  unsigned long long limit_ns;  // of a wait for a tile
};

constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;
constexpr int kUnitCost = 2;  // a unit's start and end, in tiles
constexpr int kMinTiles = 4;  // a warp's least share, in tiles
// Units of at most this length (2 is the unit's cost), and no more of them
// than blocks, have a block each: nothing is joined across blocks, which
// takes the time of some eight tiles of a warp.
constexpr int kApartTiles = 48;
// Units of at most this length, and no more of them than warps, have a warp
// each: nothing is joined at all.  22 slots x 32 heads of 96, 64 tokens: fp16
// 9.8 us, split like longer ones 12.4, bf16 10.4 and 12.9; 64 slots x 8 kv heads
// of 128, 60 tokens: 10.1 and 14.2, 11.2 and 15.1.  At 128 tokens the split is
// ahead by a tenth.
constexpr int kWholeTiles = 6;

// Most blocks of a unit whose parts one block joins directly.  More join in two
// steps, groups of about sqrt(n) blocks and then the groups.  One slot, 32/8
// heads of 64, 16384 tokens, bf16: 22.1 us, in one step 43.0; 64/8 heads of
// 128, 8192 tokens, fp16: 21.1 and 31.6.  8 to 16 here measure the same.
constexpr int kFlatJoin = 10;

// Thread blocks per SM, and stages of a warp's ring, by measurement.  More
// warps hide a tile's chain of instructions, more stages its loads; bf16 tiles
// take half as many instructions again.  32 slots to 4096 tokens, 32 heads of
// 64: fp16 3 x 3 89.5 us (2 x 6 120), bf16 4 x 2 98 us (3 x 3 102, 2 x 6 130).
// 32 slots to 2048, 40 heads of 128: fp16 2 x 2 109 us (2 x 3 115.5), bf16 2 x 3
// 109.5 us (2 x 2 111).  bf16 of 256 dims spills 270 to 340 bytes at 255
// registers, of 64 dims 30 to 60 at 128.
template <int DT, int DP>
__host__ __device__ constexpr int att_blocks() {
  return DP == 64 ? 3 + DT : 2;
}
template <int DT, int DP>
__host__ __device__ constexpr int att_stages() {
  return DP == 64 ? 3 - DT : DP == 128 ? 2 + DT : 1;
}
template <int DT, int DP>
__host__ __device__ constexpr int att_smem() {
  return kAttWarps * att_stages<DT, DP>() * 16 * DP * 4 + kAttWarps * 8 * DP * 4;
}

// Where warp w leaves its first (k = 0) and its last part: the latter in its ring.
template <int DT, int DP>
__device__ __forceinline__ float* piece_data(unsigned char* smem, int w, int k) {
  constexpr int kRing = att_stages<DT, DP>() * 16 * DP * 4;
  return reinterpret_cast<float*>(smem + (k ? w * kRing : kAttWarps * kRing + w * 8 * DP * 4));
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// mbarriers (one arrival each: the lane that orders a tile) and TMA boxes.
__device__ __forceinline__ void mbar_init(uint64_t* m, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(m)), "r"(count) : "memory");
}
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Orders this thread's writes to shared memory before later TMA writes there.
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* m, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(m)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* m, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(m)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for the phase of that parity, for limit_ns at most; the warp agrees.
__device__ __forceinline__ bool mbar_wait(uint64_t* m, uint32_t parity, unsigned long long limit_ns) {
  bool ok = mbar_try(m, parity);
  if (!__all_sync(~0u, ok)) {
    const unsigned long long t0 = now_ns();
    while (!__all_sync(~0u, ok = ok || mbar_try(m, parity)))
      if (__any_sync(~0u, now_ns() - t0 > limit_ns)) return false;
  }
  return true;
}
// K and V of a panel of 64 elements, from column x, of the rows from y of the
// pool's rows -> shared memory.
__device__ __forceinline__ void tma_panel(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* m) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(0), "r"(smem_u32(m))
      : "memory");
}
// The same of all panels.
__device__ __forceinline__ void tma_panels(uint32_t dst, const CUtensorMap* map, int y, uint64_t* m) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %2, %2}], [%4];" ::"r"(dst),
      "l"(map), "r"(0), "r"(y), "r"(smem_u32(m))
      : "memory");
}
// 16 bytes global -> shared, or zeros where bytes = 0 (the source is not read).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// c += a b, 16 x 16 by 16 x 8, 16-bit operands, fp32 sums.
template <int DT>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (DT == 0)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b
template <int DT>
__device__ __forceinline__ void mma0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (DT == 0)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two values as packed 16-bit parts: hi + lo (fp16), hi + lo + lo2 (bf16).
template <int DT>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo, uint32_t& lo2) {
  hi = pack_bits<DT>(x, y);
  x -= from_bits<DT>((uint16_t)hi);
  y -= from_bits<DT>((uint16_t)(hi >> 16));
  lo = pack_bits<DT>(x, y);
  if (DT == 1) {
    x -= from_bits<DT>((uint16_t)lo);
    y -= from_bits<DT>((uint16_t)(lo >> 16));
    lo2 = pack_bits<DT>(x, y);
  }
}

// Both rounded toward zero.
template <int DT>
__device__ __forceinline__ uint32_t pack_rz(float x, float y) {
  uint32_t r;
  if (DT == 0) asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  else asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
// The larger of |x| and least, with the sign of s.
__device__ __forceinline__ float at_least(float x, float least, float s) {
  return copysignf(fmaxf(fabsf(x), least), s);
}
// Two elements of q as parts: hi + lo (fp16, q scaled), hi + lo + 2 half (bf16).
// The parts of an element have its sign and are not 0 unless it is, so that
// an infinite key's product is infinite and of one sign in all of them: that
// moves q by less than 2^-36 of its head's largest element (fp16), 2^-28 of
// the element (bf16; below 2^-96 its parts may still be 0).
template <int DT>
__device__ __forceinline__ void split_q(float x, float y, uint32_t& hi, uint32_t& lo, uint32_t& half) {
  if (DT == 0) {
    if (fabsf(x) < 0x1p-24f && x != 0.f) x = copysignf(0x1p-24f, x);
    if (fabsf(y) < 0x1p-24f && y != 0.f) y = copysignf(0x1p-24f, y);
  }
  const float lx = DT == 0 ? 0x1p-24f : fabsf(x) * 0x1p-30f, ly = DT == 0 ? 0x1p-24f : fabsf(y) * 0x1p-30f;
  hi = pack_rz<DT>(x, y);
  float rx = x - from_bits<DT>((uint16_t)hi), ry = y - from_bits<DT>((uint16_t)(hi >> 16));
  if (DT == 0) {
    lo = pack_bits<DT>(at_least(rx, lx, x), at_least(ry, ly, y));
  } else {
    lo = pack_rz<DT>(at_least(rx, lx, x), at_least(ry, ly, y));
    rx -= from_bits<DT>((uint16_t)lo);
    ry -= from_bits<DT>((uint16_t)(lo >> 16));
    half = pack_bits<DT>(0.5f * at_least(rx, lx, x), 0.5f * at_least(ry, ly, y));
  }
}

// The visible tokens of a slot of n tokens, as tiles of 16 at multiples of
// 16: those of the first tokens, then those of the window.
struct Seen {
  int n, tail, first;    // visible: [0, first) and [tail, n)
  int first_tiles, tiles;
};
__device__ __forceinline__ Seen seen_of(const AttendArgs& a, int slot) {
  Seen v;
  int n = __ldg(a.len + slot);
  v.n = n < 0 || n > a.max_pages * a.page_tokens ? 0 : n;
  v.tail = a.window > 0 ? max(0, v.n - a.window) : 0;
  v.first = min(v.tail, a.sinks);
  v.first_tiles = (int)(((unsigned)v.first + 15u) >> 4);
  v.tiles = v.n ? v.first_tiles + (int)(((unsigned)v.n + 15u) >> 4) - (v.tail >> 4) : 0;
  return v;
}
// A tile on the line.
struct Cursor {
  long long pos;
  int slot, g, ht, tile;  // kv head, its head tile, tile of the unit
  Seen v;
  // even: where not 0, the length that every unit takes on the line
  __device__ __forceinline__ void advance(const AttendArgs& a, const int& even) {
    ++pos;
    if (++tile < v.tiles) return;
    tile = 0;
    pos += even ? even - v.tiles : kUnitCost;
    if (++ht < a.tiles) return;
    ht = 0;
    if (++g < a.kv_heads) return;
    g = 0;
    do {
      if (++slot >= a.slots) {  // past the end: not used any more
        pos = 1ll << 62;
        return;
      }
      v = seen_of(a, slot);
    } while (v.tiles == 0);
  }
  __device__ __forceinline__ int first_token() const {
    return (tile < v.first_tiles ? tile : (v.tail >> 4) + tile - v.first_tiles) << 4;
  }
  // the tile's first token, and its visible rows as bits
  __device__ __forceinline__ int rows_of(uint32_t& rows) const {
    const int t = first_token();
    const bool sink = tile < v.first_tiles;
    const int r1 = (sink ? v.first : v.n) - t, r0 = sink ? 0 : v.tail - t;
    rows = 0xffffu >> (16 - min(r1, 16)) & 0xffffu << max(r0, 0);
    return t;
  }
};

// `total` positions over `blocks` blocks: the first `more` take one more.
struct Line {
  long long each;
  int more;
  __device__ __forceinline__ void set(long long total, int blocks) {
    each = quotient(total, blocks);
    more = (int)(total - each * blocks);
  }
  __device__ __forceinline__ long long start(int b) const { return b * each + min(b, more); }
  __device__ __forceinline__ int block_of(long long pos) const {
    const long long head = more * (each + 1);
    return pos >= head ? more + (int)divide(pos - head, each) : (int)divide(pos, each + 1);
  }
  static __device__ __forceinline__ long long divide(long long a, long long b) {
    return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
  }
};

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void add_scaled(float4& sum, const float4& x, float f) {
  sum.x = fmaf(x.x, f, sum.x);
  sum.y = fmaf(x.y, f, sum.y);
  sum.z = fmaf(x.z, f, sum.z);
  sum.w = fmaf(x.w, f, sum.w);
}

// Four elements of an output row from its joined parts (no visible token: 0).
__device__ __forceinline__ void finish(const AttendArgs& a, size_t row, int d, const float4& sum,
                                       float top, float lsum) {
  const float inv = lsum > 0.f ? 1.f / lsum : lsum == lsum ? 0.f : lsum;
  *reinterpret_cast<float4*>(a.y + row * a.head_dim + d) =
      make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
  if (d == 0 && a.lse) a.lse[row] = (top + log2f(lsum)) * kLn2;
}

// Weight of a part beside the larger maximum: not 0, so that an infinite sum
// stays what it is (2^-126 of a finite one changes nothing).
__device__ __forceinline__ float part_weight(float below) { return fmaxf(ex2(below), 0x1p-126f); }

// Infinite values.  One meets weights' parts that are 0 or negative, and NaN is
// left of its column's sum.  Where that happened in a warp's share, a pass of
// its own over the share tells +-infinity from NaN: the loop over the tiles
// stays free of tests.  Heads whose scores hold NaN or +infinity stay NaN.  One
// infinite channel in every value of a layer: 346 us for 32 slots x 40 heads
// of 128 where finite ones take 109, 850 us for 8 slots to 131072 tokens (302).
template <int DT>
struct Unit {  // (slot, kv head, head tile)
  const AttendArgs& a;
  int slot, g, ht, rows;
  Seen v;
  const float* q;
  __device__ Unit(const AttendArgs& a, int slot, int g, int ht)
      : a(a), slot(slot), g(g), ht(ht), rows(min(8, a.group - ht * 8)), v(seen_of(a, slot)),
        q(a.q + ((size_t)slot * a.heads + g * a.group + ht * 8) * a.head_dim) {}
  // The visible tokens [first, end) of tile i; returns the tile's first position.
  __device__ int rows_of(int i, int& first, int& end) const {
    const bool sink = i < v.first_tiles;
    const int t = (sink ? i : (v.tail >> 4) + i - v.first_tiles) << 4;
    first = sink ? 0 : max(0, v.tail - t);
    end = min(16, (sink ? v.first : v.n) - t);
    return t;
  }
  // Key of a token in the pool; null where its page is out of range.
  __device__ const uint16_t* key_of(int t) const {
    const int page = __ldg(a.table + (size_t)slot * a.max_pages + t / a.page_tokens);
    if ((unsigned)page >= (unsigned)a.pages) return nullptr;
    return a.pool + (((size_t)page * 2 * a.kv_heads + g) * a.page_tokens + t % a.page_tokens) * a.head_dim;
  }
  __device__ bool is_new(int t) const { return a.k_new && t == v.n - 1; }
  // Element d of a token's key or value, a new one as it is stored.
  __device__ float element(bool value, int t, const uint16_t* key, int d) const {
    if (is_new(t))
      return from_bits<DT>(to_bits<DT>(__ldg((value ? a.v_new : a.k_new) +
                                             ((size_t)slot * a.kv_heads + g) * a.head_dim + d)));
    return from_bits<DT>(__ldg(key + (value ? (size_t)a.kv_heads * a.page_tokens * a.head_dim : 0) + d));
  }
  __device__ bool finite_key(int t, const uint16_t* key) const {
    bool ok = !is_new(t);  // a new one is not looked at: its score is computed
    constexpr uint32_t kTop = DT == 0 ? 0x7c00u : 0x7f80u;
#pragma unroll 1
    for (int e = 0; e < a.head_dim && ok; e += 8) {
      const uint4 k = __ldg(reinterpret_cast<const uint4*>(key + e));
      for (uint32_t w : {k.x, k.y, k.z, k.w}) ok = ok && (w & kTop) != kTop && (w >> 16 & kTop) != kTop;
    }
    return ok;
  }
  __device__ float score(int h, int t, const uint16_t* key) const {
    float s = 0.f;
#pragma unroll 1
    for (int e = 0; e < a.head_dim; ++e)
      s = fmaf(__ldg(q + h * a.head_dim + e), element(false, t, key, e), s);
    return s * a.scale;
  }
};

// A part: the tiles [i0, i1) of a unit; head h's element d is at
// to[h stride + d], or swizzled as the warps' parts are.  l: the heads' sums of
// weights (NaN where a score is NaN or +infinity); null: found from the keys.
template <int DT>
__device__ __forceinline__ void part_infinities(const Unit<DT>& u, int i0, int i1, float* to, int stride,
                                                bool swizzled, const float* l) {
  const int lane = threadIdx.x & 31, D = u.a.head_dim;
  auto at = [&](int h, int d) { return to + h * stride + (swizzled ? ((d >> 3 ^ h) << 3) + (d & 7) : d); };
  auto each_token = [&](auto f) {  // the lanes' tokens: half a warp per tile
#pragma unroll 1
    for (int i = i0 + (lane >> 4); i < i1; i += 2) {
      int r0, r1;
      const int t = u.rows_of(i, r0, r1) + (lane & 15);
      if ((lane & 15) < r0 || (lane & 15) >= r1) continue;
      if (const uint16_t* key = u.key_of(t)) f(t, key);
    }
    __syncwarp();
  };
  uint32_t odd_q = 0, closed = 0;  // heads, as bits: with a query that is not finite; that stay
#pragma unroll 1
  for (int h = 0; h < u.rows; ++h) {
#pragma unroll 1
    for (int e = lane; e < D; e += 32)
      if (!(fabsf(__ldg(u.q + h * D + e)) < INFINITY)) odd_q |= 1u << h;
    if (l && l[h] != l[h]) closed |= 1u << h;
  }
  odd_q = __reduce_or_sync(~0u, odd_q);
  // heads of `of` whose score of the token may not be finite
  auto doubtful = [&](int t, const uint16_t* key, uint32_t of) {
    return of & (u.finite_key(t, key) ? odd_q : ~0u);
  };
  if (!l) {
    each_token([&](int t, const uint16_t* key) {
      const uint32_t look = doubtful(t, key, ~closed);
#pragma unroll 1
      for (int h = 0; h < u.rows; ++h)
        if (look >> h & 1u && !(u.score(h, t, key) < INFINITY)) closed |= 1u << h;
    });
    closed = __reduce_or_sync(~0u, closed);
  }
  for (int d0 = 0; d0 < D; d0 += 32) {
    uint32_t nans = 0;  // of column d0 + lane
#pragma unroll 1
    for (int h = 0; h < u.rows && d0 + lane < D; ++h)
      if (*at(h, d0 + lane) != *at(h, d0 + lane)) nans |= 1u << h;
    nans &= ~closed;
    for (uint32_t columns = __ballot_sync(~0u, nans != 0); columns; columns &= columns - 1) {
      const int from = __ffs(columns) - 1, d = d0 + from;
      const uint32_t open = __shfl_sync(~0u, nans, from);
      uint32_t pos = 0, neg = 0, nan = 0;
      each_token([&](int t, const uint16_t* key) {
        const float x = u.element(true, t, key, d);
        if (fabsf(x) < INFINITY) return;
        uint32_t none = 0;  // heads whose score is -infinity: 0 x infinity
        const uint32_t look = doubtful(t, key, open);
#pragma unroll 1
        for (int h = 0; h < u.rows; ++h)
          if (look >> h & 1u && u.score(h, t, key) == -INFINITY) none |= 1u << h;
        nan |= x != x ? open : none;
        (x > 0.f ? pos : neg) |= open & ~none;
      });
      pos = __reduce_or_sync(~0u, pos);
      neg = __reduce_or_sync(~0u, neg);
      nan = __reduce_or_sync(~0u, nan) | (pos & neg);
      if ((open & ~nan & (pos | neg)) >> lane & 1u) *at(lane, d) = pos >> lane & 1u ? INFINITY : -INFINITY;
    }
  }
}

// Where a warp's share begins, and whether one of its sums is NaN.
struct Start {
  long long pos;
  int slot, unit, tile, odd;
};
// Goes through a warp's share.  l: [2][8], of its parts of units shared with
// other warps.
template <int DT, int DP>
__device__ __forceinline__ void infinite_values(const AttendArgs& a, const Start& from, long long share0,
                                             long long share1, int even, unsigned char* smem, const float* l) {
  const int g = from.unit / a.tiles, D = a.head_dim;
  Cursor c{from.pos, from.slot, g, from.unit - g * a.tiles, from.tile, seen_of(a, from.slot)};
  for (; c.pos < share1; c.advance(a, even)) {
    const int left = c.v.tiles - c.tile, n = share1 - c.pos < left ? (int)(share1 - c.pos) : left;
    const bool begins = c.pos - c.tile >= share0, whole = begins && n == left;
    part_infinities(Unit<DT>(a, c.slot, c.g, c.ht), c.tile, c.tile + n,
                    whole ? a.y + ((size_t)c.slot * a.heads + c.g * a.group + c.ht * 8) * D
                          : piece_data<DT, DP>(smem, threadIdx.x >> 5, begins),
                    whole ? D : DP, !whole, whole ? nullptr : l + 8 * begins);
    c.tile += n - 1;
    c.pos += n - 1;
  }
}

// A warp's part of a unit that it shares with other warps.
struct Piece {
  long long at;  // line position of the unit's first tile, -1: none
  int slot, g, ht, tiles;
};

// The parts to join: n of them, of blocks base, base + stride, ...
struct Join {
  const Piece* pc;
  int b0, nb, each, groups;  // the unit's blocks; those of a group; groups (0: none)
  int base, stride, n;
};

// DP: elements of a staged row, DK of them used by the products.  BR: rows of
// a box (16 too where tiles are gathered).  LOSE: the first tile of
// block 0 is never ordered (the self-test of the wait that runs out).
template <int DT, int DP, int DK, int BR, bool LOSE>
__global__ void __launch_bounds__(kAttThreads, att_blocks<DT, DP>())
    attend_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap map) {
  constexpr int S = att_stages<DT, DP>();
  constexpr int kTile = 16 * DP * 2;       // bytes of a tile of K (or V)
  // A stage: [16 / BR boxes][DP / 64 panels][K, V][BR rows][64 elements].
  constexpr int kValues = BR * 128, kPanel = 2 * kValues, kBox = DP / 64 * kPanel;
  auto row_at = [](int r) { return r / BR * kBox + r % BR * 128; };
  constexpr int kPieces = DP / 8;          // 16-byte pieces of a staged row
  constexpr float kShift = 14.f;  // fp16: weights are relative to a maximum less kShift
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint32_t s_mask[kAttWarps][S];
  __shared__ __align__(8) uint64_t s_bar[kAttWarps][S];
  __shared__ float s_m[kAttWarps][2][8], s_l[kAttWarps][2][8];
  __shared__ Piece s_piece[kAttWarps][2];
  __shared__ int s_even;
  // Where the warps' shares begin, until they are done; then the joins.  The
  // static memory stays within 1 KB: more of it costs a block per SM.
  __shared__ union {
    Start start[kAttWarps];
    Join join[2];
  } s_both;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = a.head_dim, P = a.page_tokens;
  const int units = a.kv_heads * a.tiles;
  auto piece_data = [&](int w, int k) { return pis::piece_data<DT, DP>(smem, w, k); };
  if (lane < 2) s_piece[warp][lane].at = -1;
  if (lane < S) mbar_init(&s_bar[warp][lane], 1);
  fence_mbar_init();
  __syncwarp();
  pdl_enter();

  // The warp's share of the line.  Lane t sums the slots [t k, t k + k).
  long long total, share0, share1;
  int grid;
  Line line{};
  Cursor cc;  // the tile being computed
  {
    int most = 0;  // the longest unit
    bool apart = false, whole = false;
    auto unit_len = [&](int tiles) { return tiles ? apart ? most : tiles + kUnitCost : 0; };
    auto scan = [&](long long v) {  // sums up to and with this lane
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long w = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += w;
      }
      return v;
    };
    const int k = (a.slots + 31) >> 5;
    long long mine = 0;
    int used = 0;
    for (int s = lane * k; s < min(a.slots, lane * k + k); ++s) {
      const int n = unit_len(seen_of(a, s).tiles);
      mine += n;
      used += n > 0;
      most = max(most, n);
    }
    most = (int)__reduce_max_sync(~0u, (uint32_t)most);
    const int per = (int)__reduce_add_sync(~0u, (uint32_t)used) * units;  // units in use
    grid = gridDim.x;
    if (most <= kApartTiles && per <= grid) {
      // a block per unit, its tiles shared evenly by the block's warps
      apart = true;
      grid = per;
    } else if (most <= kWholeTiles && per <= grid * kAttWarps) {
      // a warp per unit
      apart = whole = true;
    }
    if (apart) mine = (long long)used * most;
    if (tid == 0) s_even = whole ? most : 0;
    __syncthreads();
    long long upto = scan(mine);
    total = __shfl_sync(~0u, upto, 31) * units;
    if (!apart && total < (long long)grid * kAttWarps * kMinTiles) {
      // few tiles: if it can be, a multiple of the units, so that equal units
      // begin at a block's start and need no join across blocks
      grid = ((int)total + kAttWarps * kMinTiles - 1) / (kAttWarps * kMinTiles);
      if (per > 0 && per <= (int)gridDim.x) {
        const int up = (grid + per - 1) / per * per;
        if (up <= (int)gridDim.x) grid = up;
      }
      // no empty share between two warps of one unit
      if (grid > 1 && total < (long long)grid * kAttWarps) grid = max(1, (int)total / kAttWarps);
    }
    cc.pos = share0 = share1 = 0;
    if ((int)blockIdx.x < grid) {
      line.set(total, grid);
      const long long from = line.start(blockIdx.x), n = line.start(blockIdx.x + 1) - from;
      share0 = apart ? from : from + (warp * n) / kAttWarps;
      share1 = from + ((warp + 1) * n) / kAttWarps;
      if (whole) {
        const long long w = (long long)blockIdx.x * kAttWarps + warp, warps = (long long)grid * kAttWarps;
        share0 = quotient(w * per, (int)warps) * most;
        share1 = quotient((w + 1) * per, (int)warps) * most;
      }
      // its first slot, and where that begins
      long long at = (upto - mine) * units;
      int slot = 31 - __clz(__ballot_sync(~0u, mine > 0 && at <= share0));
      at = __shfl_sync(~0u, at, slot);
      if (k > 1) {
        const int s = slot * k + lane;
        const long long n = lane < k && s < a.slots ? unit_len(seen_of(a, s).tiles) : 0;
        const long long from = at + (scan(n) - n) * units;
        const int j = 31 - __clz(__ballot_sync(~0u, n > 0 && from <= share0));
        at = __shfl_sync(~0u, from, j);
        slot = slot * k + j;
      }
      cc.slot = slot;
      cc.v = seen_of(a, slot);
      const int len = unit_len(cc.v.tiles);
      const int unit = (int)quotient(share0 - at, len);
      const int r = (int)(share0 - at - (long long)unit * len);
      cc.g = unit / a.tiles;
      cc.ht = unit - cc.g * a.tiles;
      cc.tile = max(0, r - kUnitCost);
      cc.pos = share0 + max(0, kUnitCost - r);
      if (whole) {
        cc.tile = 0;
        cc.pos = share0;
      } else if (apart) {  // warps past the last tile have none
        const int t = cc.v.tiles, each = t / kAttWarps, more = t % kAttWarps;
        share1 = line.start(blockIdx.x + 1) - t;
        cc.tile = warp * each + min(warp, more);
        cc.pos = share0 = share1 + cc.tile;
        share1 += (warp + 1) * each + min(warp + 1, more);
      }
    }
  }
  Cursor lc = cc;  // the tile being loaded
  if (lane == 0) s_both.start[warp] = Start{cc.pos, cc.slot, cc.g * a.tiles + cc.ht, cc.tile, 0};

  const uint32_t ring = smem_u32(smem) + warp * S * 2 * kTile;
  const int pieces = D >> 3;
  const bool one_page = P % BR == 0;  // a box lies in one page
  const size_t v_off = (size_t)a.kv_heads * P * D;

  // The tile that lc points at: visible rows, first token, the row within its
  // page (of lane r's row where a tile may span pages), page number.  Where
  // it may not, lane i holds the page of box i of the unit's tiles from page0.
  uint32_t next_rows = 0;
  int next_t = 0, next_row = 0, next_page = 0, pages32 = 0, page0 = 0;
  auto page_index = [&](int t) { return a.page_shift >= 0 ? t >> a.page_shift : t / P; };
  constexpr int kBoxes = 16 / BR;  // of a tile
  auto fetch = [&](bool unit_begins) {
    if (unit_begins) {  // bring the unit's query rows near: they are read when its first tile is
      const int rows = min(8, a.group - lc.ht * 8);
      const char* q = reinterpret_cast<const char*>(
          a.q + ((size_t)lc.slot * a.heads + lc.g * a.group + lc.ht * 8) * D);
      for (int e = lane * 128; e < rows * D * 4; e += 32 * 128) {
        float unused;
        asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(unused) : "l"(q + e));
      }
    }
    next_t = lc.rows_of(next_rows);
    const int* row = a.table + (size_t)lc.slot * a.max_pages;
    if (one_page) {
      if (BR == 16) next_row = next_t - page_index(next_t) * P;
      if (unit_begins || lc.tile - page0 == 32 / kBoxes) {
        page0 = lc.tile;
        Cursor c = lc;
        c.tile += lane / kBoxes;
        pages32 = -1;
        if (c.tile < c.v.tiles) {
          uint32_t seen = 1;
          int t = BR == 16 ? c.first_token() : c.rows_of(seen);
          if (BR == 8) {  // a box may hold nothing visible, and its entry no page
            t += 8 * (lane & 1);
            seen = seen >> (8 * (lane & 1)) & 0xffu;
          }
          if (seen) pages32 = __ldg(row + page_index(t));
        }
      }
    } else {
      const int t = next_t + (lane & 15), j = page_index(t);
      next_row = t - j * P;
      next_page = next_rows >> (lane & 15) & 1u ? __ldg(row + j) : -1;
    }
  };
  // Sends that tile into a stage.  Piece pc of row r lies in panel pc / 8 at
  // piece (pc ^ r) & 7 of its row.
  constexpr int kRows = 32 / kPieces;  // rows per instruction of the gather: 4, 2, 1
  auto order = [&](uint32_t to, int y, uint64_t* bar) {  // a box
    if (a.tma == 2) {
      tma_panels(to, &map, y, bar);
    } else {
#pragma unroll 1
      for (int c = 0; c < DP / 64; ++c) tma_panel(to + c * kPanel, &map, 64 * c, y, bar);
    }
  };
  auto issue = [&](int stage) {
    const uint32_t k0 = ring + stage * 2 * kTile;
    uint64_t* bar = &s_bar[warp][stage];
    if constexpr (BR == 8) {
      const int i = 2 * (lc.tile - page0);
      const int p[2] = {__shfl_sync(~0u, pages32, i), __shfl_sync(~0u, pages32, i + 1)};
      const bool ok[2] = {(unsigned)p[0] < (unsigned)a.pages, (unsigned)p[1] < (unsigned)a.pages};
      if (lane == 0) {
        const uint32_t rows = next_rows & ((ok[0] ? 0xffu : 0u) | (ok[1] ? 0xff00u : 0u));
        if (rows != next_rows) set_status(a.status, PI_ERR_INDEX);
        s_mask[warp][stage] = rows;
        mbar_expect(bar, (ok[0] + ok[1]) * kBox);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (ok[h]) {
            const int t = next_t + 8 * h;
            order(k0 + h * kBox, (p[h] * 2 * a.kv_heads + lc.g) * P + t - page_index(t) * P, bar);
          }
      }
      return;
    }
    if (one_page) next_page = __shfl_sync(~0u, pages32, lc.tile - page0);
    const bool ok = (unsigned)next_page < (unsigned)a.pages;
    uint32_t rows = next_rows;  // rows to read: visible, and in a page
    if (one_page)
      rows = ok ? rows : 0;
    else
      rows &= __ballot_sync(~0u, ok);
    if (lane == 0) {
      if (rows != next_rows) set_status(a.status, PI_ERR_INDEX);
      s_mask[warp][stage] = rows;
    }
    const long long row = ok ? ((long long)next_page * 2 * a.kv_heads + lc.g) * P + next_row : 0;
    if (a.tma) {
      if (lane == 0) {
        if (LOSE && blockIdx.x == 0 && warp == 0 && lc.pos == cc.pos) return;  // its first tile
        mbar_expect(bar, rows ? kBox : 0);
        if (rows) order(k0, (int)row, bar);
      }
      return;
    }
    // the new token's row comes from k_new / v_new when the tile is used
    if (a.k_new && next_t < lc.v.n && lc.v.n - next_t <= 16) rows &= ~(1u << (lc.v.n - 1 - next_t));
    const int pc = lane % kPieces;
#pragma unroll 2
    for (int i = 0; i < DP / 16; ++i) {
      const int r = lane / kPieces + i * kRows;
      long long src = row + r;
      if (!one_page) src = __shfl_sync(~0u, row, r);
      if (pc < pieces) {
        const bool take = rows >> r & 1u;
        const uint16_t* p = a.pool + (take ? (size_t)src * D + 8 * pc : 0);
        const uint32_t to = k0 + (pc >> 3) * kPanel + row_at(r) + (((pc ^ r) & 7) << 4);
        cp16(to, p, take ? 16 : 0);
        cp16(to + kValues, p + (take ? v_off : 0), take ? 16 : 0);
      }
    }
    cp_commit();
  };

  if (D < DP && !a.tma)  // the padding: zeros that no copy overwrites
    for (int e = lane; e < S * 2 * kTile / 16; e += 32)
      *reinterpret_cast<uint4*>(smem + warp * S * 2 * kTile + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
  __syncwarp();
  if (lc.pos < share1) fetch(true);

  uint32_t qf[DK / 16][4], qf2[DK / 16][2];
  float o[DK / 8][2], m, l, unit_scale;
  bool fresh = true;
  int ahead = 0, load_stage = 0, stage = 0;
  uint32_t parity = 0;
  bool late = false;
  while (cc.pos < share1) {
    if (lc.pos < share1) {
      issue(load_stage);
      lc.advance(a, s_even);
      if (lc.pos < share1) fetch(lc.tile == 0);
    } else if (!a.tma) {
      cp_commit();  // an empty group: the count below stays the same
    }
    load_stage = load_stage == S - 1 ? 0 : load_stage + 1;
    if (ahead < S - 1) {  // fill the ring first
      ++ahead;
      continue;
    }

    const int g = cc.g, ht = cc.ht;
    if (fresh) {  // a unit begins: its query heads
      fresh = false;
      const int h = ht * 8 + (lane >> 2);
      const float* q = a.q + ((size_t)cc.slot * a.heads + g * a.group + min(h, a.group - 1)) * D;
      float2 f[DK / 16][2];
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = ks * 16 + e * 8 + 2 * (lane & 3);
          f[ks][e] = h < a.group && d < D ? __ldg(reinterpret_cast<const float2*>(q + d))
                                          : make_float2(0.f, 0.f);
          top = fmaxf(top, fmaxf(fabsf(f[ks][e].x), fabsf(f[ks][e].y)));
        }
      float up = 1.f;
      unit_scale = a.scale;
      if (DT == 0) {
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        // exact powers of two; 0, subnormals and infinities are clamped
        const int ex = min(max((int)(__float_as_uint(top) >> 23), 14), 254) - 127 - 13;
        up = __uint_as_float((uint32_t)(127 - ex) << 23);
        unit_scale = a.scale * __uint_as_float((uint32_t)(127 + ex) << 23);
      }
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          split_q<DT>(f[ks][e].x * up, f[ks][e].y * up, qf[ks][2 * e], qf[ks][2 * e + 1],
                      qf2[ks][e]);
      m = -INFINITY;
      l = 0.f;
#pragma unroll
      for (int j = 0; j < DK / 8; ++j) o[j][0] = o[j][1] = 0.f;
    }

    if (a.tma) {
      if (!mbar_wait(&s_bar[warp][stage], parity, a.limit_ns)) {
        set_status(a.status, PI_ERR_TIMEOUT);
        late = true;
        break;
      }
    } else {
      cp_wait<S - 1>();
    }
    __syncwarp();

    const uint32_t k0 = ring + stage * 2 * kTile, v0 = k0 + kValues;
    const uint32_t mask = s_mask[warp][stage];
    if (a.tma && mask != 0xffffu && mask != 0) {
      // values of rows that are not visible: 0 x NaN is not 0
      for (int e = lane; e < 16 * kPieces; e += 32)
        if (!(mask >> (e >> 3 & 15) & 1u))
          *reinterpret_cast<uint4*>(smem + (warp * S + stage) * 2 * kTile + (e >> 7) * kPanel + kValues +
                                    row_at(e >> 3 & 15) + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_async();
      __syncwarp();
    }
    if (a.k_new) {
      uint32_t rows;
      const int t = cc.rows_of(rows);
      const int r = cc.v.n - 1 - t;
      if (r >= 0 && r < 16 && (mask >> r & 1u)) {
        // the new token: rounded into the stage, and into its page once
        const int pg = __ldg(a.table + (size_t)cc.slot * a.max_pages + (t + r) / P);
        uint16_t* dst = a.pool + (((size_t)pg * 2 * a.kv_heads + g) * P + (t + r) % P) * D;
        for (int e = lane; e < 2 * pieces; e += 32) {
          const int kind = e >= pieces, pc = kind ? e - pieces : e;
          const float4* src = reinterpret_cast<const float4*>(
              (kind ? a.v_new : a.k_new) + ((size_t)cc.slot * a.kv_heads + g) * D) + 2 * pc;
          const float4 x = __ldg(src), y = __ldg(src + 1);
          const uint4 w = make_uint4(pack_bits<DT>(x.x, x.y), pack_bits<DT>(x.z, x.w),
                                     pack_bits<DT>(y.x, y.y), pack_bits<DT>(y.z, y.w));
          *reinterpret_cast<uint4*>(smem + (warp * S + stage) * 2 * kTile + kind * kValues +
                                    (pc >> 3) * kPanel + row_at(r) + (((pc ^ r) & 7) << 4)) = w;
          if (ht == 0) *reinterpret_cast<uint4*>(dst + kind * v_off + 8 * pc) = w;
        }
        fence_async();
        __syncwarp();
      }
    }

    if (mask) {
      // scores of 16 tokens
      // [0], [1]: even and odd steps, shorter chains (bf16 of 64 dims has no
      // registers for both); [2]: bf16's third part, whose small sums would be cut
      // beside the large ones (errors of y 0.4e-6 to 0.5e-6, in one sum 0.7e-6 to
      // 1.2e-6)
      constexpr int kChains = DT == 1 && DP == 64 ? 1 : 2;
      float sc[2][3][4];
      {
        const int r = (lane & 7) + ((lane >> 4) << 3), pc = (lane >> 3) & 1;
        const uint32_t at = k0 + row_at(r) + ((pc ^ (r & 7)) << 4);
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          uint32_t b[4];
          ldsm4(b, (at ^ ((ks & 3) << 5)) + (ks >> 2) * kPanel);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              float(&c)[4] = sc[nt][ks % kChains];
              if (ks < kChains)
                mma0<DT>(c, qf[ks], b[2 * nt], b[2 * nt + 1]);
              else
                mma<DT>(c, qf[ks], b[2 * nt], b[2 * nt + 1]);
              if (DT == 1) {
                const uint32_t q2[4] = {qf2[ks][0], qf2[ks][0], qf2[ks][1], qf2[ks][1]};
                if (ks == 0)
                  mma0<DT>(sc[nt][2], q2, b[2 * nt], b[2 * nt + 1]);
                else
                  mma<DT>(sc[nt][2], q2, b[2 * nt], b[2 * nt + 1]);
              }
            }
        }
      }
      uint32_t pf[4], pf2[2];
      float corr;
      float s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float(&c)[3][4] = sc[e >> 1];
        constexpr int k2 = kChains == 2 ? 1 : 2;
        s[e] = (c[0][e & 1] + c[k2][e & 1]) + (c[0][2 + (e & 1)] + c[k2][2 + (e & 1)]);
        if (DT == 1 && kChains == 2) s[e] += c[2][e & 1] + c[2][2 + (e & 1)];
      }
      const uint32_t mine = mask >> (2 * (lane & 3));  // rows of s: bits 0, 1, 8, 9
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = mask == 0xffffu || (mine >> ((e >> 1) * 8 + (e & 1)) & 1u) ? s[e] * unit_scale
                                                                          : -INFINITY;
      float mx = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3]));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
      // From the rounded scores, and rounded up: exponents are at most kShift
      // however large the scores are.
      if (DT == 0) mx = __fsub_ru(mx, kShift);
      const float mn = fmaxf(m, mx);
      const float ref = mn == -INFINITY ? 0.f : mn;
      corr = ex2(m - ref);
      m = mn;
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = ex2(w[e] - ref);
      l = fmaf(l, corr, (p[0] + p[1]) + (p[2] + p[3]));
      split2<DT>(p[0], p[1], pf[0], pf[1], pf2[0]);
      split2<DT>(p[2], p[3], pf[2], pf[3], pf2[1]);
      // weighted values; each tile's product is rounded once into the fp32 sums
      const int r = (lane & 7) + (((lane >> 3) & 1) << 3), pc = lane >> 4;
      const uint32_t at = v0 + row_at(r) + ((pc ^ (r & 7)) << 4);
#pragma unroll
      for (int jj = 0; jj < DK / 16; ++jj) {
        uint32_t b[4];
        ldsm4t(b, (at ^ ((jj & 3) << 5)) + (jj >> 2) * kPanel);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float c[4];
            mma0<DT>(c, pf, b[2 * u], b[2 * u + 1]);
            if (DT == 1) {
              const uint32_t p2[4] = {0u, pf2[0], 0u, pf2[1]};
              mma<DT>(c, p2, b[2 * u], b[2 * u + 1]);
            }
            o[2 * jj + u][0] = fmaf(o[2 * jj + u][0], corr, c[0] + c[2]);
            o[2 * jj + u][1] = fmaf(o[2 * jj + u][1], corr, c[1] + c[3]);
          }
      }
    }

    const long long at = cc.pos - cc.tile;  // the unit on the line: [at, at + tiles)
    const bool ends = cc.tile + 1 == cc.v.tiles;
    if (ends || cc.pos + 1 == share1) {
      const bool begins = at >= share0;
      const int h = lane >> 2;
      const int hq = ht * 8 + h;  // head of the kv head
      float lt = l;
      lt += __shfl_xor_sync(~0u, lt, 1);
      lt += __shfl_xor_sync(~0u, lt, 2);
      if (begins && ends) {
        const size_t row = (size_t)cc.slot * a.heads + g * a.group + hq;
        if (hq < a.group) {
          const float inv = lt > 0.f ? 1.f / lt : lt == lt ? 0.f : lt;
          float* y = a.y + row * D + 2 * (lane & 3);
#pragma unroll
          for (int j = 0; j < DK / 8; ++j)
            if (8 * j < D)
              *reinterpret_cast<float2*>(y + 8 * j) = make_float2(o[j][0] * inv, o[j][1] * inv);
          if ((lane & 3) == 0) {
            if (a.lse) a.lse[row] = (m + log2f(lt)) * kLn2;
          }
        }
      } else {
        const int k = begins ? 1 : 0;
        if (k) {  // into the ring, now idle
          cp_wait<0>();
          __syncwarp();
        }
        if (hq < a.group) {
          float* data = piece_data(warp, k) + h * DP + 2 * (lane & 3);
#pragma unroll
          for (int j = 0; j < DK / 8; ++j)
            *reinterpret_cast<float2*>(data + ((j ^ h) << 3)) = make_float2(o[j][0], o[j][1]);
        }
        if ((lane & 3) == 0) {
          s_m[warp][k][h] = m;
          s_l[warp][k][h] = lt;
        }
        if (lane == 0) s_piece[warp][k] = Piece{at, cc.slot, g, ht, cc.v.tiles};
      }
      float any = 0.f;
#pragma unroll
      for (int j = 0; j < DK / 8; ++j) any += o[j][0] + o[j][1];
      if (any != any) s_both.start[warp].odd = 1;
      fresh = true;
    }
    cc.advance(a, s_even);
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
    __syncwarp();  // the stage may be overwritten
  }
  // After a wait that ran out: the copies under way land before the block ends.
  for (int i = 0; late && i < S && (i == 0 || stage != load_stage); ++i) {
    mbar_wait(&s_bar[warp][stage], parity, 2000000000ull);
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
  }

  // Infinite values: once more through the share's parts.
  __syncwarp();
  if (s_both.start[warp].odd && !late)
    infinite_values<DT, DP>(a, s_both.start[warp], share0, share1, s_even, smem, s_l[warp][0]);

  // Units shared by warps.  A unit's warps within the block: the one that
  // begins it (piece 1) or the block's first (piece 0), then the followers'
  // pieces 0.  Units that other blocks share too (at most one that came in,
  // one that goes on) are left as one part for the block, and joined by the
  // last block that arrives.  A warp joins a row of a unit at a time.
  cp_wait<0>();
  __syncthreads();
  const int prow = D + 4;
  const long long block_end = line.start(blockIdx.x + 1);
  bool crossing = false;
  // lane k + 1 looks at the group that warp k's piece 1 (k = -1: piece 0 of
  // warp 0) begins; lane w at whether warp w's piece 0 goes on with it
  const long long begun = lane <= kAttWarps ? s_piece[max(lane - 1, 0)][lane > 0].at : -1;
  const long long head = lane < kAttWarps ? s_piece[lane][0].at : -1;
  uint32_t groups = __ballot_sync(~0u, begun >= 0);
  for (int turn = warp; groups; ++turn, groups &= groups - 1) {
    const int k = __ffs(groups) - 2, w0 = max(k, 0);
    const long long at = __shfl_sync(~0u, begun, k + 1);
    // warps w0 + 1, ... as long as they go on with the unit
    const uint32_t same = __ballot_sync(~0u, lane > w0 && head == at);
    const int w1 = w0 + __ffs((int)~(same >> (w0 + 1)));
    const Piece& pc = s_piece[w0][k >= 0];
    const bool local = k >= 0 && at + pc.tiles <= block_end;
    crossing |= !local;
    const int rows = min(8, a.group - pc.ht * 8);
    const size_t out0 = (size_t)pc.slot * a.heads + pc.g * a.group + pc.ht * 8;
    const int w = lane & (kAttWarps - 1);  // the lane's warp: its statistics
    const bool in = w >= w0 && w < w1;
    for (int hr = turn & (kAttWarps - 1); hr < rows; hr += kAttWarps) {
      const float mw = in ? s_m[w][w == k][hr] : -INFINITY, lw = in ? s_l[w][w == k][hr] : 0.f;
      float top = fmaxf(mw, __shfl_xor_sync(~0u, mw, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      const float f = part_weight(mw - (top == -INFINITY ? 0.f : top));
      float lsum = lw * f;
      lsum += __shfl_xor_sync(~0u, lsum, 1);
      lsum += __shfl_xor_sync(~0u, lsum, 2);
      float fw[kAttWarps];
#pragma unroll
      for (int i = 0; i < kAttWarps; ++i) fw[i] = __shfl_sync(~0u, f, i);
#pragma unroll 1
      for (int d = 4 * lane; d < D; d += 128) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f), v[kAttWarps];
        const int at_d = hr * DP + (((d >> 3) ^ (hr & 7)) << 3) + (d & 7);
#pragma unroll
        for (int i = 0; i < kAttWarps; ++i)
          if (i >= w0 && i < w1) v[i] = *reinterpret_cast<const float4*>(piece_data(i, i == k) + at_d);
#pragma unroll
        for (int i = 0; i < kAttWarps; ++i)
          if (i >= w0 && i < w1) add_scaled(sum, v[i], fw[i]);
        if (local) {
          finish(a, out0 + hr, d, sum, top, lsum);
        } else {
          float* pr = a.part + (((size_t)blockIdx.x * 2 + (k >= 0)) * 8 + hr) * prow;
          __stcg(reinterpret_cast<float4*>(pr + d), sum);
          if (d == 0) __stcg(reinterpret_cast<float2*>(pr + D), make_float2(top, lsum));
        }
      }
    }
  }
  Join(&s_join)[2] = s_both.join;
  // Releases the block's parts, which the barrier ordered before it, and
  // acquires the other blocks'.  True for the last of `of`.
  auto arrive = [](int* counter, int of) {
    int n;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
    if (n != of - 1) return false;
    *counter = 0;
    return true;
  };
  if (tid < 2) {  // 0: the unit that came in, 1: the one that goes on
    const Piece* pc = &s_piece[0][0];
    if (tid) {
      pc = &s_piece[kAttWarps - 1][1];
      for (int w = kAttWarps - 2; w >= 0 && pc->at < 0; --w) pc = &s_piece[w][1];
      if (pc->at + pc->tiles <= block_end) pc = &s_piece[0][0];
    }
    Join& jn = s_join[tid];
    jn.pc = pc;
    jn.nb = 0;
    if (pc->at >= 0 && (pc == &s_piece[0][0]) == (tid == 0)) {
      jn.b0 = line.block_of(pc->at);
      jn.nb = line.block_of(pc->at + pc->tiles - 1) - jn.b0 + 1;
    }
  }
  if (__syncthreads_or(crossing)) {
    if (tid < 2 && s_join[tid].nb) {
      Join& jn = s_join[tid];
      const int nb = jn.nb;
      jn.stride = 1;
      if (nb <= kFlatJoin) {
        jn.groups = 0;
        jn.base = jn.b0;
        jn.n = arrive(a.arrived + jn.b0, nb) ? nb : 0;
      } else {
        // Groups of about sqrt(nb), none of one block: so a counter at each
        // group's second block is no other unit's.
        const int each = (int)ceilf(sqrtf((float)nb));
        int groups = (nb + each - 1) / each;
        groups -= nb - (groups - 1) * each == 1;
        const int i = min(((int)blockIdx.x - jn.b0) / each, groups - 1);
        const int size = i == groups - 1 ? nb - i * each : each;
        jn.each = each;
        jn.groups = groups;
        jn.base = jn.b0 + i * each;
        jn.n = arrive(a.arrived + kAttendGrid + jn.base + 1, size) ? size : 0;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
      if (s_join[x].nb == 0) continue;
      const Join& jn = s_join[x];
      const Piece& pc = *jn.pc;
      const int rows = min(8, a.group - pc.ht * 8), vecs = D >> 2, items = rows * vecs;
      const size_t out0 = (size_t)pc.slot * a.heads + pc.g * a.group + pc.ht * 8;
      // Where block b left its part; a group its own, in the second place of
      // its first block, or in that of the unit's second block: both blocks
      // lie within the unit, so no other unit's part is there.
      auto part_of = [&](int b, bool group) {
        const int begins = b == jn.b0;
        return a.part + (size_t)(group ? 2 * (b + begins) + 1 : 2 * b + begins) * (8 * prow);
      };
#pragma unroll 1
      while (jn.n) {
        const int n = jn.n, base = jn.base, stride = jn.stride;
        const bool last = jn.groups == 0;
        // two items of a thread together, four parts at a time: their reads overlap
#pragma unroll 1
        for (int e = tid; e < items; e += 2 * kAttThreads) {
          float4 sum[2];
          float top[2], lsum[2];
          int hr[2], d[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = min(e + i * kAttThreads, items - 1);
            hr[i] = at / vecs;
            d[i] = 4 * (at - hr[i] * vecs);
            sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            top[i] = -INFINITY;
            lsum[i] = 0.f;
          }
#pragma unroll 1
          for (int j0 = 0; j0 < n; j0 += 4) {
            float4 v[2][4];
            float2 q[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (j0 + j < n) {  // the (j0 + j)-th part
                  const float* pr = part_of(base + (j0 + j) * stride, stride > 1) + hr[i] * prow;
                  q[i][j] = __ldcg(reinterpret_cast<const float2*>(pr + D));
                  v[i][j] = __ldcg(reinterpret_cast<const float4*>(pr + d[i]));
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (j0 + j < n) {
                  const float up = fmaxf(top[i], q[i][j].x), ref = up == -INFINITY ? 0.f : up;
                  const float was = part_weight(top[i] - ref), is = part_weight(q[i][j].x - ref);
                  sum[i] = make_float4(sum[i].x * was, sum[i].y * was, sum[i].z * was, sum[i].w * was);
                  add_scaled(sum[i], v[i][j], is);
                  lsum[i] = fmaf(lsum[i], was, q[i][j].y * is);
                  top[i] = up;
                }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (e + i * kAttThreads >= items) break;
            if (last) {
              finish(a, out0 + hr[i], d[i], sum[i], top[i], lsum[i]);
            } else {
              float* to = part_of(base, true) + hr[i] * prow;
              __stcg(reinterpret_cast<float4*>(to + d[i]), sum[i]);
              if (d[i] == 0) __stcg(reinterpret_cast<float2*>(to + D), make_float2(top[i], lsum[i]));
            }
          }
        }
        if (last) break;
        __syncthreads();
        if (tid == 0) {
          Join& next = s_join[x];
          next.n = arrive(a.arrived + next.b0, next.groups) ? next.groups : 0;
          next.base = next.b0;
          next.stride = next.each;
          next.groups = 0;
        }
        __syncthreads();
      }
    }
  }

  // Empty slots, and lengths out of range.
  for (int s = blockIdx.x; s < a.slots; s += gridDim.x) {
    const int n = __ldg(a.len + s);
    if (n > 0 && n <= a.max_pages * P) continue;
    if (n != 0 && tid == 0) set_status(a.status, PI_ERR_INDEX);
    for (int e = tid; e < a.heads * D; e += kAttThreads) a.y[(size_t)s * a.heads * D + e] = 0.f;
    if (a.lse)
      for (int e = tid; e < a.heads; e += kAttThreads) a.lse[(size_t)s * a.heads + e] = -INFINITY;
  }
}

// A thread stores N pieces of eight elements, 256 pieces apart, of the line
// (token, K or V, kv head, piece): all its reads are under way before the
// first store.  Bound: HBM bandwidth (fp32 rows in, 16-bit rows out).  N = 4
// for prompts (12001 tokens of 32 heads of 128: 97 us, 90 % of the measured
// copy rate; N = 1: 104.7; 8 bytes spill at 64 registers), 1 where N = 4 would
// leave SMs without a block (32 tokens of 40 heads, in a graph: 1.7 us against
// 3.1).

struct AppendArgs {
  const float *k, *v;
  const int *slot, *pos, *table;
  uint16_t* pool;  // the layer's pages
  int* status;
  long long total;  // pieces
  int kv_heads, head_dim, page_tokens, pages, slots, max_pages;
};

template <int DT, int N>
__global__ void __launch_bounds__(256, 4) append_kernel(const AppendArgs a) {
  pdl_enter();
  const int pieces = a.head_dim >> 3, half = a.kv_heads * pieces;
  for (long long e0 = blockIdx.x * (256ll * N) + threadIdx.x; e0 < a.total;
       e0 += gridDim.x * (256ll * N)) {
    float4 f[N][2];
    int s[N], p[N], r[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const long long e = e0 + u * 256;
      s[u] = -1;
      if (e >= a.total) continue;
      const int i = (int)quotient(e, 2 * half);
      r[u] = (int)(e - (long long)i * (2 * half));
      s[u] = __ldg(a.slot + i);
      p[u] = __ldg(a.pos + i);
      const bool val = r[u] >= half;
      const float4* src = reinterpret_cast<const float4*>(val ? a.v : a.k) +
                          2 * ((size_t)i * half + (r[u] - (val ? half : 0)));
      f[u][0] = __ldcs(src);
      f[u][1] = __ldcs(src + 1);
    }
    int page[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (s[u] == -1) continue;
      if ((unsigned)s[u] >= (unsigned)a.slots || p[u] < 0 || p[u] >= a.max_pages * a.page_tokens) {
        set_status(a.status, PI_ERR_INDEX);
        s[u] = -1;
        continue;
      }
      const int j = p[u] / a.page_tokens;
      page[u] = __ldg(a.table + (size_t)s[u] * a.max_pages + j);
      p[u] -= j * a.page_tokens;
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (s[u] == -1) continue;
      if (checked_page(page[u], a.pages, a.status) < 0) continue;
      const bool val = r[u] >= half;
      const int q = r[u] - (val ? half : 0), g = q / pieces;
      uint16_t* dst = a.pool + ((((size_t)page[u] * 2 + val) * a.kv_heads + g) * a.page_tokens + p[u]) *
                                   a.head_dim + 8 * (q - g * pieces);
      const float4 x = f[u][0], y = f[u][1];
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bits<DT>(x.x, x.y), pack_bits<DT>(x.z, x.w),
                                                  pack_bits<DT>(y.x, y.y), pack_bits<DT>(y.z, y.w));
    }
  }
}

// Map over a layer's rows (K and V rows of every page and kv head), 128-byte
// swizzle, box_rows rows of K and of V per box.  Head dimensions that are
// multiples of 64: {64 elements, rows, K / V, panels}, a box of all panels (a
// lane's request takes some 100 cycles to issue).  Others: {row, rows, K / V},
// a box per panel, zeros past the row's end.  False where the driver offers no
// such map.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static bool make_rows_map(CUtensorMap* m, void* base, long long rows, const pi_cache_desc& C,
                          int panels, int box_rows) {
  static const EncodeFn encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(p) : nullptr;
  }();
  if (!encode) return false;
  const cuuint64_t row = (cuuint64_t)C.head_dim * 2, half = (cuuint64_t)C.kv_heads * C.page_tokens;
  const bool whole = C.head_dim % 64 == 0;
  const cuuint64_t dims[4] = {whole ? 64u : (cuuint64_t)C.head_dim, (cuuint64_t)rows - half, 2u,
                              (cuuint64_t)C.head_dim / 64};
  const cuuint64_t strides[3] = {row, half * row, 128u};
  const cuuint32_t box[4] = {64u, (cuuint32_t)box_rows, 2u, (cuuint32_t)panels},
                   steps[4] = {1u, 1u, 1u, 1u};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, whole ? 4 : 3, base, dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Limit of a wait: 1 s, or PI_WAIT_LIMIT_NS as for the FFN kernels.
static unsigned long long wait_limit() {
  static const unsigned long long limit = [] {
    const char* e = std::getenv("PI_WAIT_LIMIT_NS");
    const unsigned long long v = e ? std::strtoull(e, nullptr, 10) : 0;
    return v >= 1000ull && v <= 10000000000ull ? v : 1000000000ull;
  }();
  return limit;
}

template <int DT, int DP, int DK, int BR, bool LOSE = false>
pi_status launch_boxes(const AttendArgs& a, const CUtensorMap& map, pi_stream stream) {
  DevInfo di;
  pi_status st = dev_info(&di);
  if (st != PI_OK) return st;
  constexpr int smem = att_smem<DT, DP>();
  st = ensure_smem(reinterpret_cast<const void*>(attend_kernel<DT, DP, DK, BR, LOSE>), smem);
  if (st != PI_OK) return st;
  // All blocks that are resident together, or fewer where the longest slots
  // that the tables and the window allow cannot use them.
  long long seen = (long long)a.max_pages * a.page_tokens;
  if (a.window > 0 && (long long)a.window + a.sinks < seen) seen = (long long)a.window + a.sinks;
  const long long units = (long long)a.slots * a.kv_heads * a.tiles;
  const long long shares = units * (seen / 16 + 3 + kUnitCost) / (kAttWarps * kMinTiles) + 1;
  const long long useful = shares > units ? shares : units;
  long long grid = di.sms * att_blocks<DT, DP>();
  if (grid > kAttendGrid) grid = kAttendGrid;
  if (grid > useful) grid = useful;
  return launch(attend_kernel<DT, DP, DK, BR, LOSE>, dim3((unsigned)grid), kAttThreads, smem, stream, a,
                map);
}

template <int DT, int DP, int DK = DP>
pi_status launch_attend(const AttendArgs& a, const CUtensorMap& map, pi_stream stream) {
  return a.tma && a.page_tokens % 16 ? launch_boxes<DT, DP, DK, 8>(a, map, stream)
                                     : launch_boxes<DT, DP, DK, 16>(a, map, stream);
}

// Shared memory holds whole panels of 64 elements; the products stop at the
// next of 80, 96 and 192, which is most of a tile's time where it is
// instructions.  32 heads, 16 slots to 4096 tokens: heads of 80 67 us in fp16
// and 74 in bf16 (as 128: 75, 84), of 96 70 and 77 (75, 84); 16 heads of 192
// 69 and 77 (as 256: 73, 92).
template <int DT>
pi_status launch_dims(const AttendArgs& a, const CUtensorMap& map, pi_stream stream) {
  if (a.head_dim <= 64) return launch_attend<DT, 64>(a, map, stream);
  if (a.head_dim <= 80) return launch_attend<DT, 128, 80>(a, map, stream);
  if (a.head_dim <= 96) return launch_attend<DT, 128, 96>(a, map, stream);
  if (a.head_dim <= 128) return launch_attend<DT, 128>(a, map, stream);
  if (a.head_dim <= 192) return launch_attend<DT, 256, 192>(a, map, stream);
  return launch_attend<DT, 256>(a, map, stream);
}

}  // namespace pis

using namespace pis;

static pi_status attention(const pi_cache_desc* cache, int32_t layer, int32_t slots,
                           int32_t heads, int32_t max_pages, const float* q,
                           const float* k_new, const float* v_new, const int32_t* table,
                           const int32_t* len, void* pool, float scale, int32_t window,
                           int32_t sinks, float* y, float* lse, int32_t* dev_status, void* ws,
                           size_t ws_bytes, pi_stream stream, unsigned long long lose_ns) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  const pi_cache_desc& C = *cache;
  st = check_slots(C, slots, max_pages);
  if (st != PI_OK) return st;
  if (layer < 0 || layer >= C.layers || heads < 1 || heads > kMaxHeads || heads % C.kv_heads)
    return PI_ERR_SHAPE;
  if (window < 0 || sinks < 0) return PI_ERR_SHAPE;
  if (!q || !table || !len || !pool || !y || !dev_status || !ws || !k_new != !v_new)
    return PI_ERR_NULL;
  if (!all_aligned(q, k_new, v_new, table, len, pool, y, lse, dev_status, ws)) return PI_ERR_ALIGN;
  if (ws_bytes < cache_ws(C, slots, heads).total) return PI_ERR_WORKSPACE;
  const CacheWs w = cache_ws(C, slots, heads);
  AttendArgs a{};
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.table = table;
  a.len = len;
  a.pool = static_cast<uint16_t*>(pool) + (size_t)layer * C.pages * page_elems(C);
  a.y = y;
  a.lse = lse;
  a.status = dev_status;
  a.arrived = reinterpret_cast<int*>(static_cast<char*>(ws) + w.arrived);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + w.part);
  a.slots = slots;
  a.heads = heads;
  a.kv_heads = C.kv_heads;
  a.group = heads / C.kv_heads;
  a.head_dim = C.head_dim;
  a.page_tokens = C.page_tokens;
  a.pages = C.pages;
  a.page_shift = C.page_tokens & (C.page_tokens - 1) ? -1 : __builtin_ctz((unsigned)C.page_tokens);
  a.max_pages = max_pages;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale * 1.4426950408889634f;
  const long long rows = (long long)C.pages * 2 * C.kv_heads * C.page_tokens;
  CUtensorMap map = {};
  a.limit_ns = wait_limit();
  const int panels = C.head_dim <= 64 ? 1 : C.head_dim <= 128 ? 2 : 4;
  a.tma = C.page_tokens % 8 == 0 && C.head_dim >= 64 && rows < (1ll << 31) &&
          make_rows_map(&map, a.pool, rows, C, panels, C.page_tokens % 16 ? 8 : 16);
  if (a.tma && C.head_dim % 64 == 0) a.tma = 2;
  a.tiles = (a.group + 7) / 8;
  if (lose_ns) {
    if (C.dtype != PI_F16 || C.head_dim != 64 || a.tma != 2 || C.page_tokens % 16) return PI_ERR_SHAPE;
    a.limit_ns = lose_ns;
    return launch_boxes<0, 64, 64, 16, true>(a, map, stream);
  }
  return C.dtype == PI_F16 ? launch_dims<0>(a, map, stream) : launch_dims<1>(a, map, stream);
}

extern "C" {

size_t pi_cache_workspace_size(const pi_cache_desc* cache, int32_t slots, int32_t heads) {
  if (check_cache(cache) != PI_OK || slots < 1 || slots > PI_CACHE_MAX_SLOTS) return 0;
  if (heads < 0 || heads > kMaxHeads || heads % cache->kv_heads) return 0;
  return cache_ws(*cache, slots, heads).total;
}

pi_status pi_paged_attention(const pi_cache_desc* cache, int32_t layer, int32_t slots,
                             int32_t heads, int32_t max_pages, const float* q,
                             const float* k_new, const float* v_new, const int32_t* table,
                             const int32_t* len, void* pool, float scale, int32_t window,
                             int32_t sinks, float* y, float* lse, int32_t* dev_status, void* ws,
                             size_t ws_bytes, pi_stream stream) {
  return attention(cache, layer, slots, heads, max_pages, q, k_new, v_new, table, len, pool, scale,
                   window, sinks, y, lse, dev_status, ws, ws_bytes, stream, 0);
}

pi_status pi_selftest_attention_timeout(const pi_cache_desc* cache, int32_t slots, int32_t heads,
                                        int32_t max_pages, const float* q, const int32_t* table,
                                        const int32_t* len, void* pool, float* y,
                                        int32_t* dev_status, void* ws, size_t ws_bytes,
                                        int64_t limit_ns, pi_stream stream) {
  if (limit_ns < 1000 || limit_ns > 5000000000LL) return PI_ERR_SHAPE;
  return attention(cache, 0, slots, heads, max_pages, q, nullptr, nullptr, table, len, pool, 1.f, 0, 0,
                   y, nullptr, dev_status, ws, ws_bytes, stream, (unsigned long long)limit_ns);
}

pi_status pi_cache_append(const pi_cache_desc* cache, int32_t layer, int32_t slots,
                          int32_t max_pages, int32_t tokens, const int32_t* slot,
                          const int32_t* pos, const float* k, const float* v,
                          const int32_t* table, void* pool, int32_t* dev_status,
                          pi_stream stream) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  const pi_cache_desc& C = *cache;
  st = check_slots(C, slots, max_pages);
  if (st != PI_OK) return st;
  if (layer < 0 || layer >= C.layers || tokens < 0) return PI_ERR_SHAPE;
  if (!table || !pool || !dev_status) return PI_ERR_NULL;
  if (tokens > 0 && (!slot || !pos || !k || !v)) return PI_ERR_NULL;
  if (!all_aligned(slot, pos, k, v, table, pool, dev_status)) return PI_ERR_ALIGN;
  if (tokens == 0) return PI_OK;
  AppendArgs a{k, v, slot, pos, table,
               static_cast<uint16_t*>(pool) + (size_t)layer * C.pages * page_elems(C), dev_status,
               2ll * tokens * C.kv_heads * (C.head_dim / 8), C.kv_heads, C.head_dim, C.page_tokens,
               C.pages, slots, max_pages};
  DevInfo di;
  st = dev_info(&di);
  if (st != PI_OK) return st;
  const bool many = a.total >= 1024ll * di.sms;
  const long long blocks = many ? (a.total + 1023) / 1024 : (a.total + 255) / 256;
  const bool f16 = C.dtype == PI_F16;
  return launch(many ? (f16 ? append_kernel<0, 4> : append_kernel<1, 4>)
                     : (f16 ? append_kernel<0, 1> : append_kernel<1, 1>),
                dim3((unsigned)(blocks < 65536 ? blocks : 65536)), 256, 0, stream, a);
}

}  // extern "C"
