// attend.cu — attention of one new token per slot over a paged cache, and
// the stores of new keys and values (include/pi_serve.h).
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
// third part.  fp16's narrow exponent range is met by exact powers of two:
// q is scaled to [2^13, 2^14) per head, p by 2^14.
//
// Work split.  All visible tokens of all (slot, kv head, group of heads)
// units, in blocks of 64 tokens, form one line; each thread block takes an
// equal contiguous share of it, found from the lengths on the device, so
// ragged lengths balance and nothing depends on the host knowing them.  A
// unit that spans thread blocks leaves partial results; the last of its
// blocks to arrive joins them in block order (no waiting; order fixed).
//
// Data flow.  A warp owns every fourth 16-token tile of its block's share
// and streams it through its own ring of cp.async stages (no block-wide
// barrier per tile); page numbers are fetched one tile ahead of their use;
// rows outside the visible set are never read (zero-filled).
struct AttendArgs {
  const float *q, *k_new, *v_new;
  const int *table, *len;
  uint16_t* pool;  // the layer's pages
  float *y, *lse;
  int* status;
  int* arrived;   // [kAttendGrid] arrivals at the units that begin in a block
  float* part;    // [grid][2][heads of a unit][head_dim + 4]: o, m, l of split units
  int slots, heads, kv_heads, group, head_dim, page_tokens, pages, max_pages, window, sinks;
  int tiles;      // head tiles per kv head: ceil(group / (8 MT))
  int min_blocks; // least 64-token blocks of a thread block
  float scale;    // scale log2(e)
};

constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;

// Stages of a warp's ring: two thread blocks per SM (one at 256 dims).
template <int DP>
__host__ __device__ constexpr int att_stages() {
  return DP == 64 ? 6 : 3;
}
template <int DP>
__host__ __device__ constexpr int att_smem() {
  return kAttWarps * att_stages<DP>() * 16 * DP * 4 + kAttWarps * 8 * DP * 4;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
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
__device__ __forceinline__ int blocks_of(int tiles) {
  return (tiles + kAttWarps - 1) / kAttWarps;
}

// A position on the line of 64-token blocks.
struct Cursor {
  int slot, unit, blk, blocks;  // unit: kv head x head tiles
  Seen v;
  __device__ __forceinline__ void enter(const AttendArgs& a, int s) {
    slot = s;
    v = seen_of(a, s);
    blocks = blocks_of(v.tiles);
  }
  __device__ __forceinline__ void advance(const AttendArgs& a) {
    if (++blk < blocks) return;
    blk = 0;
    if (++unit < a.kv_heads * a.tiles) return;
    unit = 0;
    do {
      if (slot + 1 >= a.slots) return;  // past the end: not used any more
      enter(a, slot + 1);
    } while (blocks == 0);
  }
  // first token of the warp's tile, and the tile's visible rows [r0, r1)
  __device__ __forceinline__ int tile(int warp, int& r0, int& r1) const {
    const int i = blk * kAttWarps + warp;
    if (i < v.first_tiles) {
      r0 = 0;
      r1 = min(16, v.first - 16 * i);
      return 16 * i;
    }
    const int t = ((v.tail >> 4) + i - v.first_tiles) << 4;
    r0 = max(0, v.tail - t);
    r1 = i < v.tiles ? min(16, v.n - t) : 0;
    return t;
  }
};

template <int DT, int DP, int MT>
__global__ void __launch_bounds__(kAttThreads, DP == 256 ? 1 : 2) attend_kernel(const AttendArgs a) {
  constexpr int S = att_stages<DP>();
  constexpr int kTile = 16 * DP * 2;       // bytes of a tile of K (or V)
  constexpr int kRow = DP * 2;             // bytes of a staged row
  constexpr int kPieces = DP / 8;          // 16-byte pieces of a staged row
  constexpr float kShift = DT == 0 ? 14.f : 0.f;  // weights carry 2^kShift
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[kAttWarps];
  __shared__ int s_slot0, s_last;
  __shared__ long long s_before;
  __shared__ uint32_t s_mask[kAttWarps][S];
  __shared__ float s_m[kAttWarps][8], s_l[kAttWarps][8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = a.head_dim, P = a.page_tokens;
  const int units = a.kv_heads * a.tiles;
  float* part = reinterpret_cast<float*>(smem + kAttWarps * S * 2 * kTile);
  pdl_enter();

  // Empty slots, and lengths out of range.
  for (int s = blockIdx.x; s < a.slots; s += gridDim.x) {
    const int n = __ldg(a.len + s);
    if (n > 0 && n <= a.max_pages * P) continue;
    if (n != 0 && tid == 0) set_status(a.status, PI_ERR_INDEX);
    for (int e = tid; e < a.heads * D; e += kAttThreads) a.y[(size_t)s * a.heads * D + e] = 0.f;
    if (a.lse)
      for (int e = tid; e < a.heads; e += kAttThreads) a.lse[(size_t)s * a.heads + e] = -INFINITY;
  }

  // This block's share of the line.  Thread t holds the slots [t k, t k + k).
  long long share0, share1, total;
  int grid;
  {
    const int k = (a.slots + kAttThreads - 1) / kAttThreads;
    long long mine = 0;
    for (int s = tid * k; s < min(a.slots, tid * k + k); ++s) mine += blocks_of(seen_of(a, s).tiles);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long w = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += w;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    long long before = upto - mine;
    total = 0;
    for (int w = 0; w < kAttWarps; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    total *= units;
    const long long most = (total + a.min_blocks - 1) / a.min_blocks;
    grid = (int)(most < (long long)gridDim.x ? most : (long long)gridDim.x);
    if ((int)blockIdx.x >= grid) return;
    share0 = blockIdx.x * total / grid;
    share1 = (blockIdx.x + 1) * total / grid;
    // the thread whose slots hold share0 looks for it there
    long long at = before * units;
    if (at <= share0 && share0 < at + mine * units) {
      for (int s = tid * k;; ++s) {
        const long long n = (long long)blocks_of(seen_of(a, s).tiles) * units;
        if (share0 < at + n) {
          s_slot0 = s;
          s_before = at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
  }
  const int steps = (int)(share1 - share0);
  Cursor cc;  // the block being computed
  cc.enter(a, s_slot0);
  cc.unit = (int)((share0 - s_before) / cc.blocks);
  cc.blk = (int)((share0 - s_before) % cc.blocks);
  long long unit_at = share0 - cc.blk;  // where the unit begins on the line
  Cursor lc = cc;  // the block being loaded

  const uint32_t ring = smem_u32(smem) + warp * S * 2 * kTile;
  const int pieces = D >> 3, ksteps = (D + 15) >> 4;
  const bool one_page = (P & 15) == 0;  // a tile lies in one page
  const size_t v_off = (size_t)a.kv_heads * P * D;

  // Page number of the tile that lc points at (lane r: of its row r).
  auto fetch = [&]() -> int {
    int r0, r1;
    const int t = lc.tile(warp, r0, r1) + (one_page ? 0 : lane & 15);
    const bool use = one_page ? r1 > 0 : (lane & 15) >= r0 && (lane & 15) < r1;
    return use ? __ldg(a.table + (size_t)lc.slot * a.max_pages + t / P) : -2;
  };
  // Sends the tile at lc into a stage.
  auto issue = [&](int stage, int page) {
    int r0, r1;
    const int t = lc.tile(warp, r0, r1);
    const int g = lc.unit / a.tiles;
    const bool ok = (unsigned)page < (unsigned)a.pages;
    if (!ok && page != -2) set_status(a.status, PI_ERR_INDEX);
    uint32_t mask = 0;  // rows to read: visible, and in a page
    if (r1 > r0) mask = (0xffffu >> (16 - r1)) & (0xffffu << r0);
    if (one_page)
      mask = ok ? mask : 0;
    else
      mask &= __ballot_sync(~0u, ok);
    if (lane == 0) s_mask[warp][stage] = mask;
    // the new token's row comes from k_new / v_new when the tile is used
    if (a.k_new && t < lc.v.n && lc.v.n - t <= 16) mask &= ~(1u << (lc.v.n - 1 - t));
    const long long row =
        ok ? ((long long)page * 2 * a.kv_heads + g) * P + (one_page ? t : t + (lane & 15)) % P : 0;
    const uint32_t k0 = ring + stage * 2 * kTile;
    const int pc = lane % kPieces;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const int r = lane / kPieces + i * (32 / kPieces);
      long long src = row + r;
      if (!one_page) src = __shfl_sync(~0u, row, r);
      if (pc < 2 * ksteps) {
        const bool take = (mask >> r & 1u) && pc < pieces;
        const uint16_t* p = a.pool + (take ? (size_t)src * D + 8 * pc : 0);
        const uint32_t dst = k0 + r * kRow + ((pc ^ (r & 7)) << 4);
        cp16(dst, p, take ? 16 : 0);
        cp16(dst + kTile, p + (take ? v_off : 0), take ? 16 : 0);
      }
    }
  };

  int issued = 0;
  int page = steps > 0 ? fetch() : -2;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    if (issued < steps) {
      issue(i, page);
      if (++issued < steps) {
        lc.advance(a);
        page = fetch();
      }
    }
    cp_commit();
  }

  uint32_t qf[MT][DP / 16][4], qf2[DT == 1 ? MT : 1][DP / 16][2];
  float o[MT][DP / 8][2], m[MT], l[MT], unit_scale[MT];
  int seg0 = cc.blk;  // the segment's first block in its unit
  bool fresh = true;

  for (int i = 0; i < steps; ++i) {
    cp_wait<S - 2>();
    __syncwarp();
    if (issued < steps) {
      issue((i + S - 1) % S, page);
      if (++issued < steps) {
        lc.advance(a);
        page = fetch();
      }
    }
    cp_commit();

    const int g = cc.unit / a.tiles, ht = cc.unit % a.tiles;
    if (fresh) {  // a unit begins: its query heads
      fresh = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int h = (ht * MT + mt) * 8 + (lane >> 2);
        const float* q = a.q + ((size_t)cc.slot * a.heads + g * a.group + min(h, a.group - 1)) * D;
        float2 f[DP / 16][2];
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = ks * 16 + e * 8 + 2 * (lane & 3);
            f[ks][e] = h < a.group && d < D ? __ldg(reinterpret_cast<const float2*>(q + d))
                                            : make_float2(0.f, 0.f);
            top = fmaxf(top, fmaxf(fabsf(f[ks][e].x), fabsf(f[ks][e].y)));
          }
        float up = 1.f;
        unit_scale[mt] = a.scale;
        if (DT == 0) {
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          // exact powers of two; 0, subnormals and infinities are clamped
          const int ex = min(max((int)(__float_as_uint(top) >> 23), 14), 254) - 127 - 13;
          up = __uint_as_float((uint32_t)(127 - ex) << 23);
          unit_scale[mt] = a.scale * __uint_as_float((uint32_t)(127 + ex) << 23);
        }
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            split2<DT>(f[ks][e].x * up, f[ks][e].y * up, qf[mt][ks][2 * e], qf[mt][ks][2 * e + 1],
                       qf2[DT == 1 ? mt : 0][ks][e]);
        m[mt] = -INFINITY;
        l[mt] = 0.f;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) o[mt][j][0] = o[mt][j][1] = 0.f;
      }
    }

    const int stage = i % S;
    const uint32_t k0 = ring + stage * 2 * kTile, v0 = k0 + kTile;
    const uint32_t mask = s_mask[warp][stage];
    if (a.k_new) {
      int r0, r1;
      const int t = cc.tile(warp, r0, r1);
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
          *reinterpret_cast<uint4*>(smem + (warp * S + stage) * 2 * kTile + kind * kTile + r * kRow +
                                    ((pc ^ (r & 7)) << 4)) = w;
          if (ht == 0) *reinterpret_cast<uint4*>(dst + kind * v_off + 8 * pc) = w;
        }
        __syncwarp();
      }
    }

    if (mask) {
      // scores of 16 tokens
      float sc[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
      {
        const int r = (lane & 7) + ((lane >> 4) << 3), pc = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
          if (ks >= ksteps) break;
          uint32_t b[4];
          ldsm4(b, k0 + r * kRow + (((2 * ks + pc) ^ (r & 7)) << 4));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma<DT>(sc[mt][0], qf[mt][ks], b[0], b[1]);
            mma<DT>(sc[mt][1], qf[mt][ks], b[2], b[3]);
            if (DT == 1) {
              const uint32_t q2[4] = {0u, qf2[mt][ks][0], 0u, qf2[mt][ks][1]};
              mma<DT>(sc[mt][0], q2, b[0], b[1]);
              mma<DT>(sc[mt][1], q2, b[2], b[3]);
            }
          }
        }
      }
      uint32_t pf[MT][4], pf2[MT][2];
      float corr[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float s[4], mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = (e >> 1) * 8 + 2 * (lane & 3) + (e & 1);
          s[e] = sc[mt][e >> 1][e & 1] + sc[mt][e >> 1][2 + (e & 1)];
          if (!(mask >> tok & 1u)) s[e] = -INFINITY;
          else mx = fmaxf(mx, s[e] * unit_scale[mt]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
        const float mn = fmaxf(m[mt], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;
        corr[mt] = ex2(m[mt] - ref);
        m[mt] = mn;
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = (e >> 1) * 8 + 2 * (lane & 3) + (e & 1);
          p[e] = mask >> tok & 1u ? ex2(fmaf(s[e], unit_scale[mt], kShift - ref)) : 0.f;
        }
        l[mt] = fmaf(l[mt], corr[mt], (p[0] + p[1]) + (p[2] + p[3]));
        split2<DT>(p[0], p[1], pf[mt][0], pf[mt][1], pf2[mt][0]);
        split2<DT>(p[2], p[3], pf[mt][2], pf[mt][3], pf2[mt][1]);
      }
      // weighted values; each tile's product is rounded once into the fp32 sums
      const int r = (lane & 7) + (((lane >> 3) & 1) << 3), pc = lane >> 4;
#pragma unroll
      for (int jj = 0; jj < DP / 16; ++jj) {
        if (jj >= ksteps) break;
        uint32_t b[4];
        ldsm4t(b, v0 + r * kRow + (((2 * jj + pc) ^ (r & 7)) << 4));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            mma<DT>(c, pf[mt], b[2 * u], b[2 * u + 1]);
            if (DT == 1) {
              const uint32_t p2[4] = {0u, pf2[mt][0], 0u, pf2[mt][1]};
              mma<DT>(c, p2, b[2 * u], b[2 * u + 1]);
            }
            o[mt][2 * jj + u][0] = fmaf(o[mt][2 * jj + u][0], corr[mt], c[0] + c[2]);
            o[mt][2 * jj + u][1] = fmaf(o[mt][2 * jj + u][1], corr[mt], c[1] + c[3]);
          }
      }
    }

    const bool ends = cc.blk + 1 == cc.blocks;
    if (ends || i + 1 == steps) {  // the segment ends: join the warps
      const bool whole = ends && seg0 == 0;
      const int rows = min(8 * MT, a.group - ht * 8 * MT);  // query heads of the unit
      const int vecs = D >> 2;
      const int prow = D + 4;
      // slot 0: the block's share begins in this unit
      float* mine = a.part + ((size_t)blockIdx.x * 2 + (unit_at <= share0 ? 0 : 1)) * (8 * MT) * prow;
      const size_t out0 = (size_t)cc.slot * a.heads + g * a.group + ht * 8 * MT;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int live = min(8, rows - 8 * mt);
        if (live <= 0) break;
        const int h = lane >> 2;
        float lt = l[mt];
        lt += __shfl_xor_sync(~0u, lt, 1);
        lt += __shfl_xor_sync(~0u, lt, 2);
        __syncthreads();  // the previous join has been read
        if ((lane & 3) == 0) {
          s_m[warp][h] = m[mt];
          s_l[warp][h] = lt;
        }
        if (h < live) {
#pragma unroll
          for (int j = 0; j < DP / 8; ++j)
            *reinterpret_cast<float2*>(part + (warp * 8 + h) * DP + ((j ^ h) << 3) + 2 * (lane & 3)) =
                make_float2(o[mt][j][0], o[mt][j][1]);
        }
        __syncthreads();
        for (int e = tid; e < live * vecs; e += kAttThreads) {
          const int hh = e / vecs, d = 4 * (e % vecs);
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, s_m[w][hh]);
          const float ref = top == -INFINITY ? 0.f : top;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
          float lsum = 0.f;
#pragma unroll
          for (int w = 0; w < kAttWarps; ++w) {
            const float f = ex2(s_m[w][hh] - ref);
            const float4 x = *reinterpret_cast<const float4*>(
                part + (w * 8 + hh) * DP + (((d >> 3) ^ hh) << 3) + (d & 7));
            sum.x = fmaf(x.x, f, sum.x);
            sum.y = fmaf(x.y, f, sum.y);
            sum.z = fmaf(x.z, f, sum.z);
            sum.w = fmaf(x.w, f, sum.w);
            lsum = fmaf(s_l[w][hh], f, lsum);
          }
          const int hr = 8 * mt + hh;
          if (whole) {
            const float inv = lsum > 0.f ? 1.f / lsum : lsum == lsum ? 0.f : lsum;
            *reinterpret_cast<float4*>(a.y + (out0 + hr) * D + d) =
                make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
            if (d == 0 && a.lse)
              a.lse[out0 + hr] = (top + (log2f(lsum) - kShift)) * 0.6931471805599453f;
          } else {
            float* pr = mine + (size_t)hr * prow;
            __stcg(reinterpret_cast<float4*>(pr + d), sum);
            if (d == 0) {
              __stcg(pr + D, top);
              __stcg(pr + D + 1, lsum);
            }
          }
        }
      }
      if (!whole) {
        // the unit's blocks on the line, and the thread blocks that hold them
        const long long end = unit_at + cc.blocks;
        const int b0 = (int)(((unit_at + 1) * grid - 1) / total);
        const int b1 = (int)((end * grid - 1) / total);
        __threadfence();
        __syncthreads();
        if (tid == 0) s_last = atomicAdd(a.arrived + b0, 1) == b1 - b0;
        __syncthreads();
        if (s_last) {
          __threadfence();
          if (tid == 0) a.arrived[b0] = 0;
          const int slot0 = unit_at <= b0 * total / grid ? 0 : 1;
          for (int e = tid; e < rows * vecs; e += kAttThreads) {
            const int hr = e / vecs, d = 4 * (e % vecs);
            auto at = [&](int b) {
              return a.part + (((size_t)b * 2 + (b == b0 ? slot0 : 0)) * (8 * MT) + hr) * prow;
            };
            float top = -INFINITY;
            for (int b = b0; b <= b1; ++b) top = fmaxf(top, __ldcg(at(b) + D));
            const float ref = top == -INFINITY ? 0.f : top;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float lsum = 0.f;
            for (int b = b0; b <= b1; ++b) {
              const float* pr = at(b);
              const float f = ex2(__ldcg(pr + D) - ref);
              const float4 x = __ldcg(reinterpret_cast<const float4*>(pr + d));
              sum.x = fmaf(x.x, f, sum.x);
              sum.y = fmaf(x.y, f, sum.y);
              sum.z = fmaf(x.z, f, sum.z);
              sum.w = fmaf(x.w, f, sum.w);
              lsum = fmaf(__ldcg(pr + D + 1), f, lsum);
            }
            const float inv = lsum > 0.f ? 1.f / lsum : lsum == lsum ? 0.f : lsum;
            *reinterpret_cast<float4*>(a.y + (out0 + hr) * D + d) =
                make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
            if (d == 0 && a.lse)
              a.lse[out0 + hr] = (top + (log2f(lsum) - kShift)) * 0.6931471805599453f;
          }
        }
      }
      fresh = true;
      seg0 = 0;
      if (ends) unit_at += cc.blocks;
    }
    if (i + 1 < steps) cc.advance(a);
  }
}

// Thread = eight elements of one (token, K or V, kv head) row.
template <int DT>
__global__ void __launch_bounds__(256) append_kernel(const float* k, const float* v,
                                                     const int* slot, const int* pos,
                                                     const int* table, uint16_t* pool,
                                                     long long total, int kv_heads, int head_dim,
                                                     int page_tokens, int pages, int slots,
                                                     int max_pages, int* status) {
  pdl_enter();
  const int pieces = head_dim >> 3;
  for (long long e = blockIdx.x * 256ll + threadIdx.x; e < total; e += gridDim.x * 256ll) {
    const int pc = (int)(e % pieces);
    const long long r = e / pieces;  // (token, kind, head)
    const int g = (int)(r % kv_heads);
    const long long tk = r / kv_heads;
    const int kind = (int)(tk & 1);
    const int i = (int)(tk >> 1);
    const int s = slot[i], p = pos[i];
    if (s == -1) continue;
    if (s < 0 || s >= slots || p < 0 || p >= max_pages * page_tokens) {
      set_status(status, PI_ERR_INDEX);
      continue;
    }
    const int page = checked_page(table[(size_t)s * max_pages + p / page_tokens], pages, status);
    if (page < 0) continue;
    const float4* src = reinterpret_cast<const float4*>((kind ? v : k) +
                                                        ((size_t)i * kv_heads + g) * head_dim) + 2 * pc;
    const float4 f0 = src[0], f1 = src[1];
    uint16_t* dst = pool + ((((size_t)page * 2 + kind) * kv_heads + g) * page_tokens +
                            p % page_tokens) * head_dim + 8 * pc;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bits<DT>(f0.x, f0.y), pack_bits<DT>(f0.z, f0.w),
                                                pack_bits<DT>(f1.x, f1.y), pack_bits<DT>(f1.z, f1.w));
  }
}

template <int DT, int DP, int MT>
pi_status launch_attend(const AttendArgs& a, pi_stream stream) {
  DevInfo di;
  pi_status st = dev_info(&di);
  if (st != PI_OK) return st;
  constexpr int smem = att_smem<DP>();
  st = ensure_smem(reinterpret_cast<const void*>(attend_kernel<DT, DP, MT>), smem);
  if (st != PI_OK) return st;
  const int grid = di.sms * (DP == 256 ? 1 : 2);
  return launch(attend_kernel<DT, DP, MT>, dim3((unsigned)(grid < kAttendGrid ? grid : kAttendGrid)),
                kAttThreads, smem, stream, a);
}

}  // namespace pis

using namespace pis;

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
  a.max_pages = max_pages;
  a.window = window;
  a.sinks = sinks;
  a.min_blocks = 4;
  a.scale = scale * 1.4426950408889634f;
  const bool two = att_two_tiles(C.head_dim, a.group);
  a.tiles = (a.group + (two ? 15 : 7)) / (two ? 16 : 8);
  if (C.dtype == PI_F16) {
    if (C.head_dim <= 64) return two ? launch_attend<0, 64, 2>(a, stream) : launch_attend<0, 64, 1>(a, stream);
    if (C.head_dim <= 128) return two ? launch_attend<0, 128, 2>(a, stream) : launch_attend<0, 128, 1>(a, stream);
    return launch_attend<0, 256, 1>(a, stream);
  }
  if (C.head_dim <= 64) return two ? launch_attend<1, 64, 2>(a, stream) : launch_attend<1, 64, 1>(a, stream);
  if (C.head_dim <= 128) return two ? launch_attend<1, 128, 2>(a, stream) : launch_attend<1, 128, 1>(a, stream);
  return launch_attend<1, 256, 1>(a, stream);
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
  const long long total = 2ll * tokens * C.kv_heads * (C.head_dim / 8);
  const long long blocks = (total + 255) / 256;
  uint16_t* base = static_cast<uint16_t*>(pool) + (size_t)layer * C.pages * page_elems(C);
  return launch(C.dtype == PI_F16 ? append_kernel<0> : append_kernel<1>,
                dim3((unsigned)(blocks < 152 * 64 ? blocks : 152 * 64)), 256, 0, stream, k, v, slot,
                pos, table, base, total, C.kv_heads, C.head_dim, C.page_tokens, C.pages, slots,
                max_pages, dev_status);
}

}  // extern "C"
