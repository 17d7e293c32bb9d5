// q8_attn.cu -- attention of one query token a sequence over the 8-bit paged
// cache: every position (decode_attn_q8), or a hybrid-head layer whose sparse
// heads read their sets only.
//
// Mathematics.  With c_j, c'_j the codes of key and value j and sk, sv the scales
// of their blocks: s_j = (q . c_j) sk / sqrt(d), p = softmax(s) over every j < n_b
// (or over the head's set), out = sum_j p_j sv c'_j.  A sequence of no rows and an
// empty set give zeros.  Both products run on the tensor cores without a second
// rounding of the cache, and take the scales afterwards.
//
// Numbers.  The codes become halves (exact: both code types fit 11 bits).  (The
// 8-bit form of mma.sync with q in two parts: 490 executed instructions for 16 rows
// against 415, 54 us against 52 for 131072 positions.)  q is scaled by a power of
// two that brings its largest magnitude to [2^13, 2^14): a bf16 is then a half
// exactly down to 2^-27 of the largest, and an fp32 is held in two halves (22
// bits).  The weight that multiplies the values' codes is w_j = p_j sv_j; it is what
// must fit a half, so the running reference of the online softmax is the maximum
// of s_j log2(e) + log2(sv_j), and the normaliser sums w_j / sv_j beside it.  The
// reference is kept 6 below the maximum seen and moved only when a weight would
// pass 2^15: weights down to 2^-31 of the largest keep a place in the half's range
// (an 8-bit float's range would lose the many small weights of a long context).
// A weight is held in two halves (22 bits): one alone (11 bits) moves every tenth
// bf16 output to its neighbour.
//
// Work split.  The unit is a slab of 32 rows of one KV head.  All slabs of the
// call, ordered by sequence, head and position, are cut into one equal range per
// CTA and that into one per warp, whatever the lengths (a sequence's and a head's
// slabs are a segment; a hybrid layer counts only the rows that some head of the
// group uses).  A warp works alone: it brings its slabs into a ring of its own in
// shared memory and runs the G heads of the group over each slab at once; no
// barrier joins the warps before the end.  A full slab is 32 consecutive rows: a
// TMA box of K and one of V (two each when pages have 16 rows).  The rows of sparse
// heads' sets, and a slab cut by the sequence's end, come row by row (cp.async,
// absent rows as zeros).  At the end the CTA merges its warps' states of a segment, writes what
// is complete and leaves at most two states open: of a segment that began in an
// earlier CTA and of one that goes on in a later CTA.  The second kernel merges
// those.  When there are fewer segments than CTAs and the table is narrow, every
// segment is one CTA's and nothing is left to merge.  All sums have a fixed order.
//
// Layouts.  Rows lie in shared memory with the TMA's swizzle (16-byte pieces of a
// row XORed with its number).  S = K q^T as m16n8k16 with 16 of the slab's rows as M:
// a lane takes 16-byte piece c (c = lane % 4) of its two rows; which dimension a k index means is free as long as q agrees, so a
// row's words convert to A fragments in place.  O^T = V^T P with the
// dimensions as M: a lane takes piece lane / 4 of four rows; interleaving the bytes
// of two rows gives the pairs along k that A wants.  Which row stands at which index
// of M and k is free too: index i is row i ^ 4 (i & 1), which makes both reads
// free of bank conflicts.  P moves from the accumulator layout to B by a
// transpose of 8x8 halves (movmatrix).
//
// Bound by memory where there is enough to read: 131072 positions of 8 KV heads of
// 128 (268 MB) take 49 us, of which the slabs 38 (7.1 TB/s), finding the ranges and
// the first rows 5, merging and the second launch 5.  Next to it stand the
// instructions (a 16-row step took 415 of them in slabs of 16, and less in slabs of
// 32, whose bookkeeping is shared): int8 codes, two more per pair to become halves,
// stay 8 % above the copy rate's time.  12 warps with rings of two slabs and 168
// registers (49.0 / 96 us on that case / a batch of 64 of up to 8191 in int8) beat 8
// with rings of three (49.5 / 104) and 16 of 16-row slabs (51.6 / 102).
#include <algorithm>

#include "q8.cuh"

namespace lychee {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = kQ8Warps;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = kQ8Stages;
constexpr int kRows = kQ8Slab;       // rows of a slab: two halves of 16, the M of the products
// What a segment costs beside its slabs, in slabs (256 sequences of up to 600: 40.3 us
// without it, 34.8 with 1, 35.2 with 2).
constexpr int kSegCost = 1;
constexpr float kRefBelow = 6.f;     // the reference lies this far below the maximum (log2)
constexpr float kRefSlack = 15.f;    // and moves when a weight passes it by more than this
constexpr uint32_t kAbsent = 0xffffffffu;  // of a slab's rows: none
constexpr float kNoRef = -3.402823466e38f;   // no row yet: the lowest finite number (differences of two stay numbers)
constexpr uint32_t kFullSlab = 1u << 29;   // stage header: consecutive rows, a scale a half
constexpr uint32_t kAllHeads = 1u << 30;   // ... and every head uses every row

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_u(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A box of rows from y on of the map's array, all of their bytes, to dst in the map's swizzle.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar),
      "l"(policy)
      : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <typename T>
__device__ __forceinline__ float4 load_q4(const T* p);
template <>
__device__ __forceinline__ float4 load_q4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
template <>
__device__ __forceinline__ float4 load_q4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

template <typename T, int CODE, int D, int G>
struct Cfg {
  static constexpr bool kTwoQ = sizeof(T) == 4;          // q in two halves (the weights always are)
  static constexpr bool kBeside = G <= 4;                // ... in columns 0-3 and 4-7 of one product (a q of
                                                         // one half stands in both)
  static constexpr int NQ = kTwoQ && !kBeside ? 2 : 1;   // ... or in two products
  static constexpr int NP = kBeside ? 1 : 2;
  static constexpr int KM = D / 16;                      // blocks of 16 dimensions of O
  static constexpr int H = D / 64;                       // 16-byte pieces of K a lane takes of a row
  static constexpr int VB = D / 8;                       // bytes of V a lane takes of each of its four rows
  static constexpr int DATA = 2 * kRows * D;             // a stage's rows: K, then V
  static constexpr int OFF_V = kRows * D;
  // beside the rows, per stage: row scales (K's, V's; of a full slab one per half:
  // K's, V's), the rows each head uses (a word a head), the header {segment, position
  // | flags}
  static constexpr int AUX_S = 0, AUX_META = 256, AUX_HEAD = 288, AUX = 304;
  static constexpr int WARP_AUX = kStages * AUX + 32;    // and the stages' mbarriers
  static constexpr int OFF_AUX = kWarps * kStages * DATA;
  static constexpr int STATE = G * (D + 2);              // floats of a state: m[G], l[G], acc[G][D]
  // the states that warps end on their way: behind that where they fit (else in the
  // workspace); the block's other shared variables take less than 768 bytes
  static constexpr int OFF_ENDED = OFF_AUX + kWarps * WARP_AUX;
  static constexpr bool kEndedHere = OFF_ENDED + kWarps * STATE * 4 + 1024 + 768 <= 227 * 1024;
  static constexpr int SMEM = OFF_ENDED + (kEndedHere ? kWarps * STATE * 4 : 0) + 1024;   // + alignment slack
  static_assert(WARP_AUX % 16 == 0 && kStages * 8 <= 32, "aligned");
  static_assert(DATA / 2 % 1024 == 0 || D == 64, "swizzled rows on 1024-byte (D = 64: 512-byte) boundaries");
  static_assert(kWarps * STATE * 4 <= OFF_AUX, "the states are merged where the rings were");
};

// Where a range of slabs begins.
struct Start {
  int seg, tile, slab;  // segment b * Hkv + g; hybrid: tile of the segment, slab of the tile
};

template <typename T, int CODE, int D, int G, bool HYB>
struct Warp {
  using C = Cfg<T, CODE, D, G>;
  const Q8AttnParams& p;
  uint32_t ring, aux, bars;
  int lane, r, c;
  uint32_t gathered;    // bit i: stage i was last filled row by row
  uint32_t kofs, vofs_a, vofs_b;   // this lane's pieces in a stage: K of row R, V of rows Ra and Rb

  // The warp's place in its slabs: the next one to copy.
  int seg, b, g, n;
  int at, rows;         // slab of the segment (hybrid: of the tile), rows of it
  int tile;             // hybrid (else 0)
  bool sparse, mixed;   // hybrid: the group has sparse heads only / has some
  // ... and what was loaded for it: the page (consecutive rows) or this lane's row
  uint32_t pre, pre_m;  // hybrid: the rows that head `lane` uses, or the heads that use this lane's row

  __device__ __forceinline__ Warp(const Q8AttnParams& pp, uint32_t ring_, uint32_t aux_)
      : p(pp), ring(ring_), aux(aux_), bars(aux_ + kStages * C::AUX) {
    lane = threadIdx.x & 31;
    r = lane >> 2;
    c = lane & 3;
    gathered = 0;
    const int R = r ^ ((r & 1) << 2), Ra = 2 * c, Rb = (2 * c) ^ 5;
    kofs = R * D + ((D == 128 ? c ^ (R & 7) : c ^ ((R >> 1) & 3)) << 4);
    vofs_a = C::OFF_V + Ra * D + (D == 128 ? (r ^ (Ra & 7)) << 4 : (((r >> 1) ^ ((Ra >> 1) & 3)) << 4) + (r & 1) * 8);
    vofs_b = C::OFF_V + Rb * D + (D == 128 ? (r ^ (Rb & 7)) << 4 : (((r >> 1) ^ ((Rb >> 1) & 3)) << 4) + (r & 1) * 8);
    tile = 0;
    sparse = mixed = false;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kStages; ++i)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bars + 8 * i), "r"(i == 0 && p.withhold_first ? 2 : 1)
                     : "memory");
      fence_mbar_init();
    }
    __syncwarp();
  }
  __device__ __forceinline__ bool retrieval(int h) const { return (p.role[h >> 5] >> (h & 31)) & 1u; }

  // ---- the cursor
  __device__ __forceinline__ void enter(int seg_) {
    seg = seg_;
    b = seg / p.Hkv;
    g = seg - b * p.Hkv;
    n = min(max(p.seqlens[b], 0), p.N_max);
    at = 0;
    if (HYB) {
      int kept = 0;
#pragma unroll
      for (int t = 0; t < G; ++t) kept += retrieval(g * G + t);
      sparse = kept == 0;
      mixed = kept > 0 && kept < G;
    } else {
      rows = n;
    }
  }
  // To the first segment after `seg` that has positions; false if there is none.
  __device__ __forceinline__ bool enter_next() {
    int s = seg + 1;
    while (s < p.B * p.Hkv) {
      enter(s);
      if (n > 0) return true;
      s = (b + 1) * p.Hkv;
    }
    return false;
  }
  // Hybrid: to the first tile of the segment at or after `from` that has rows; false
  // if none does.
  __device__ __forceinline__ bool enter_tile(int from) {
    for (int t0 = from; t0 * kQ8Tile < n; t0 += 32) {
      const int k = (t0 + lane) * kQ8Tile < n ? __ldcg(&p.tile_rows[(size_t)seg * p.ntiles + t0 + lane]) : 0;
      const uint32_t any = __ballot_sync(kFull, k > 0);
      if (any) {
        const int l = __ffs(any) - 1;
        tile = t0 + l;
        rows = __shfl_sync(kFull, k, l);
        at = 0;
        return true;
      }
    }
    return false;
  }
  // Start loading what the slab at the cursor needs.
  __device__ __forceinline__ void preload() {
    if (HYB && sparse) {
      const int e = kRows * at + lane;
      const size_t from = ((size_t)seg * p.ntiles + tile) * kQ8Tile + e;
      pre = kAbsent;
      pre_m = 0;
      if (e < rows) {
        pre = __ldcg(p.list_rows + from);
        pre_m = __ldcg(p.list_heads + from);
      }
    } else {
      // (a page of 16 positions is half a slab: odd lanes take the second half's)
      const int pos0 = tile * kQ8Tile + kRows * at, pos = pos0 + 16 * (lane & 1);
      pre = p.c.table[(size_t)b * p.c.max_pages + ((pos < n ? pos : pos0) >> p.c.page_log2)];
      if (HYB && mixed) {
        pre_m = 0xffffffffu;
        if (lane < G && !retrieval(g * G + lane))
          pre_m = __ldcg(p.bitmaps + ((size_t)b * p.Hq + g * G + lane) * p.nwords + (pos0 >> 5));
      }
    }
  }
  __device__ __forceinline__ bool begin(const Start& s) {
    if (s.seg >= p.B * p.Hkv) return false;
    enter(s.seg);
    if (HYB && !enter_tile(s.tile)) return false;
    at = s.slab;
    preload();
    return true;
  }
  // To the next slab; false: there is none.
  __device__ __forceinline__ bool advance() {
    if (kRows * ++at >= rows) {
      if (HYB) {
        if (!enter_tile(tile + 1)) {
          do {
            if (!enter_next()) return false;
          } while (!enter_tile(0));
        }
      } else if (!enter_next()) {
        return false;
      }
    }
    preload();
    return true;
  }
  // Hybrid: no tile before `t` has rows.
  __device__ __forceinline__ bool first_tile(int seg_, int t) const {
    for (int t0 = 0; t0 < t; t0 += 32)
      if (__any_sync(kFull, t0 + lane < t && __ldcg(&p.tile_rows[(size_t)seg_ * p.ntiles + t0 + lane]) > 0)) return false;
    return true;
  }

  // ---- the slab at the cursor into stage `si`
  __device__ __forceinline__ void copy(int si) {
    const uint32_t st = ring + si * C::DATA, ax = aux + si * C::AUX, bar = bars + 8 * si;
    const int log2p = p.c.page_log2;
    uint32_t myrow, heads, flags = 0;     // this lane's row; lane t: the rows head t uses
    if (!HYB || !sparse) {
      // consecutive positions: a half lies in one page
      const int pos0 = tile * kQ8Tile + kRows * at;
      const int rest = min(n - pos0, kRows);
      const bool ok = pre < (uint32_t)p.c.num_pages;      // of this lane's half
      if (!ok && lane < 2 && 16 * lane < rest) flag_error(p.err, kErrBadIndex);
      const int unit = (int)pre * p.Hkv + g;
      const uint32_t row0 = ((uint32_t)unit << log2p) + ((pos0 + 16 * (lane & 1)) & ((1 << log2p) - 1));
      flags = (uint32_t)pos0;
      if (rest == kRows && __all_sync(kFull, ok)) {
        if (lane < 2) {
          copy4(ax + C::AUX_S + 8 * lane, p.c.k_scale + unit);      // the halves' scales
          copy4(ax + C::AUX_S + 8 * lane + 4, p.c.v_scale + unit);
          asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        }
        const uint32_t row1 = __shfl_sync(kFull, row0, 1);          // (joins the lanes, too)
        if (lane == 0) {
          if ((gathered >> si) & 1u) fence_proxy_async_smem();   // ordinary writes before the TMA's
          sts64(ax + C::AUX_HEAD, (uint32_t)seg, flags | kFullSlab | (HYB && mixed ? 0u : kAllHeads));
          asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"((uint32_t)C::DATA)
                       : "memory");
          const uint64_t policy = l2_evict_first_policy();
          tma_rows(st, &p.tmk, (int)row0, bar, policy);
          tma_rows(st + C::OFF_V, &p.tmv, (int)row0, bar, policy);
          if (log2p == 4) {   // (boxes of 16 rows; else of 32)
            tma_rows(st + 16 * D, &p.tmk, (int)row1, bar, policy);
            tma_rows(st + C::OFF_V + 16 * D, &p.tmv, (int)row1, bar, policy);
          }
        }
        if (HYB && mixed && lane < G) sts_u(ax + C::AUX_META + 4 * lane, pre_m);
        gathered &= ~(1u << si);
        return;
      }
      // lane i: row i
      const uint32_t half0 = __shfl_sync(kFull, row0, 0), half1 = __shfl_sync(kFull, row0, 1);
      const uint32_t oks = __ballot_sync(kFull, ok);
      const bool in = lane < rest && ((oks >> (lane >> 4)) & 1u);
      myrow = in ? (lane < 16 ? half0 : half1) + (lane & 15) : kAbsent;
      heads = __ballot_sync(kFull, in) & (HYB && mixed ? pre_m : 0xffffffffu);
      if (HYB && lane < rest && !in) {
        // a position without a page ranks last in the sets that are handed on
#pragma unroll 1
        for (int t = 0; t < G; ++t)
          if (retrieval(g * G + t)) p.logits[((size_t)seg * G + t) * p.N_max + pos0 + lane] = -INFINITY;
      }
    } else {
      myrow = pre;
      heads = 0;
#pragma unroll
      for (int t = 0; t < G; ++t) {
        const uint32_t m = __ballot_sync(kFull, (pre_m >> t) & 1u);
        if (lane == t) heads = m;
      }
    }
    // row by row.  Absent rows are zeros with scale 1.
    gathered |= 1u << si;
    constexpr int LPR = D / 16, RPI = 32 / LPR;   // lanes a row, rows an instruction
    const int lr = lane / LPR, q = lane % LPR;
#pragma unroll
    for (int j = 0; j < kRows / RPI; ++j) {
      const int R = RPI * j + lr;
      const uint32_t row = __shfl_sync(kFull, myrow, R);
      const uint32_t dst = st + R * D + ((D == 128 ? q ^ (R & 7) : q ^ ((R >> 1) & 3)) << 4);
      const uint32_t from = 16 * q;
      if (row != kAbsent) {
        copy16(dst, p.c.k + ((size_t)row * D + from));
        copy16(dst + C::OFF_V, p.c.v + ((size_t)row * D + from));
      } else {
        sts128(dst, 0u, 0u, 0u, 0u);
        sts128(dst + C::OFF_V, 0u, 0u, 0u, 0u);
      }
    }
    if (myrow != kAbsent) {
      copy4(ax + C::AUX_S + lane * 4, p.c.k_scale + (myrow >> log2p));
      copy4(ax + C::AUX_S + 128 + lane * 4, p.c.v_scale + (myrow >> log2p));
    } else {
      sts_u(ax + C::AUX_S + lane * 4, __float_as_uint(1.f));
      sts_u(ax + C::AUX_S + 128 + lane * 4, __float_as_uint(1.f));
    }
    if (lane < G) sts_u(ax + C::AUX_META + 4 * lane, heads);
    if (lane == 0) sts64(ax + C::AUX_HEAD, (uint32_t)seg, flags);
    // the phase ends when every lane's copies have landed
    asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
    __syncwarp();
    if (lane == 0) asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
  }

  // ---- the heads' states
  uint32_t qf[C::NQ][C::KM][2];   // q as B fragments
  float fq[2];                    // powers of two that undo q's scaling, of this lane's two columns
  float ref[2], l[2];             // reference (log2) and sum of p, of this lane's two columns
  float acc[C::KM][4];

  __device__ __forceinline__ int column_head(int j) const { return (C::kBeside ? 2 * (c & 1) : 2 * c) + j; }

  size_t logit_row;               // hybrid: where this lane's first column's logits go
  int logit_cols;                 // ... bit j: column j is a retrieval head (written by this lane)
  bool retrieves;                 // ... the group has a retrieval head

  struct RawQ {
    float4 x[C::KM];
  };
  __device__ __forceinline__ void fetch_q(int sg, RawQ& raw) const {
    const int t = C::kBeside ? r & 3 : r;
#pragma unroll
    for (int m = 0; m < C::KM; ++m) {
      raw.x[m] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < G)
        raw.x[m] = load_q4<T>(static_cast<const T*>(p.q) + ((size_t)sg * G + t) * D + (m >> 2) * 64 +
                              16 * c + 4 * (m & 3));
    }
  }
  __device__ __forceinline__ void set_q(int sg, const RawQ& q) {
    if (HYB) {
      const int h0 = sg % p.Hkv * G;
      logit_row = ((size_t)sg * G + column_head(0)) * p.N_max;
      logit_cols = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (column_head(j) < G && (!C::kBeside || c < 2) && retrieval(h0 + column_head(j))) logit_cols |= 1 << j;
      retrieves = __any_sync(kFull, logit_cols != 0);
    }
    const float4 (&x)[C::KM] = q.x;
    float mx = 0.f;
#pragma unroll
    for (int m = 0; m < C::KM; ++m)
      mx = fmaxf(mx, fmaxf(fmaxf(fabsf(x[m].x), fabsf(x[m].y)), fmaxf(fabsf(x[m].z), fabsf(x[m].w))));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    // the largest magnitude to [2^13, 2^14) (below 2^-100 the same factor as at 2^-100)
    constexpr int top = 13;
    const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
    const float up = exp2_int(top - e);
    const float down = mx < INFINITY ? exp2_int(e - top) : NAN;   // (an infinite q has no score)
#pragma unroll
    for (int m = 0; m < C::KM; ++m) {
      const float a = x[m].x * up, bb = x[m].y * up, cc = x[m].z * up, d = x[m].w * up;
      uint32_t w0 = pack_half(a, bb), w1 = pack_half(cc, d);
      if constexpr (C::kTwoQ) {
        const float2 h0 = unpack_half(w0), h1 = unpack_half(w1);
        const uint32_t l0 = pack_half(a - h0.x, bb - h0.y), l1 = pack_half(cc - h1.x, d - h1.y);
        if constexpr (C::NQ == 2) {
          qf[1][m][0] = l0;
          qf[1][m][1] = l1;
        } else if (r >= 4) {
          w0 = l0;
          w1 = l1;
        }
      }
      qf[0][m][0] = w0;
      qf[0][m][1] = w1;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) fq[j] = __shfl_sync(kFull, down, (column_head(j) & 7) * 4);
  }
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int m = 0; m < C::KM; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
    ref[0] = ref[1] = kNoRef;
    l[0] = l[1] = 0.f;
  }

  // ---- one slab: stage `si`, its header in hd
  __device__ __forceinline__ void consume(int si, uint2 hd) {
    const uint32_t st = ring + si * C::DATA, ax = aux + si * C::AUX;
    const int R = r ^ ((r & 1) << 2);      // this lane's rows of S in a half: R and R + 8
    // ---- S of both halves
    float s[2][4];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      float s2[4] = {0.f, 0.f, 0.f, 0.f};
      s[a][0] = s[a][1] = s[a][2] = s[a][3] = 0.f;
#pragma unroll
      for (int h = 0; h < C::H; ++h) {
        const uint32_t at = (st + kofs + a * 16 * D) ^ (h << 6);
        const uint4 lo = lds128(at), hi = lds128(at + 8 * D);
        const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = h * 4 + j;
          uint32_t a0, a1, a2, a3;
          codes_to_half<CODE>(wl[j], a0, a2);
          codes_to_half<CODE>(wh[j], a1, a3);
          mma_f16((j & 1) ? s2 : s[a], a0, a1, a2, a3, qf[0][m][0], qf[0][m][1]);
          if constexpr (C::NQ == 2) mma_f16((j & 1) ? s2 : s[a], a0, a1, a2, a3, qf[1][m][0], qf[1][m][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[a][i] += s2[i];
      if (C::kTwoQ && C::kBeside) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[a][i] += __shfl_xor_sync(kFull, s[a][i], 2);
      }
    }
    // s[a][0], s[a][1]: row 16 a + R, columns 2c and 2c + 1; s[a][2], s[a][3]: row 16 a + R + 8
    float sk[2][2], lv[2][2], inv[2][2];   // [half][row]: K scale, log2 and reciprocal of V scale
    if (hd.y & kFullSlab) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const uint2 x = lds64(ax + C::AUX_S + 8 * a);
        sk[a][0] = sk[a][1] = __uint_as_float(x.x);
        lv[a][0] = lv[a][1] = fast_log2(__uint_as_float(x.y));
        inv[a][0] = inv[a][1] = fast_exp2(-lv[a][0]);
      }
    } else {
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sk[a][i] = lds_f(ax + C::AUX_S + (R + 8 * i + 16 * a) * 4);
          lv[a][i] = fast_log2(lds_f(ax + C::AUX_S + 128 + (R + 8 * i + 16 * a) * 4));
          inv[a][i] = fast_exp2(-lv[a][i]);
        }
    }
    // bit 16 a + 8 i: this lane's row counts for column j's head
    uint32_t used[2] = {0xffffffffu, 0xffffffffu};
    if (!(hd.y & kAllHeads)) {
      const uint2 x = lds64(ax + C::AUX_META + 4 * column_head(0));
      used[0] = x.x >> R;
      used[1] = x.y >> R;
    }
    // t: log2 of a row's weight times its scale, -inf where a head does not use it.
    // (Columns beyond the group's heads hold zero queries; nothing reads them.)
    float t[2][4];
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[a][2 * i + j] = s[a][2 * i + j] * sk[a][i] * fq[j];   // (the scale first: the two factors' product may overflow)
          const bool on = (used[j] >> (16 * a + 8 * i)) & 1u;
          t[a][2 * i + j] = on ? fmaf(s[a][2 * i + j], p.scale_log2, lv[a][i]) : -INFINITY;
          top[j] = fmaxf(top[j], t[a][2 * i + j]);
        }
    if (HYB && retrieves) {
      // (a group with a retrieval head has consecutive rows)
      float* out = p.logits + logit_row + ((hd.y & 0xffffffu) + R);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if ((logit_cols >> j) & 1) {
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if ((used[j] >> (16 * a + 8 * i)) & 1u) out[(size_t)j * p.N_max + 16 * a + 8 * i] = s[a][2 * i + j];
        }
    }
    if (__any_sync(kFull, top[0] > ref[0] + kRefSlack || top[1] > ref[1] + kRefSlack)) {
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = top[j];
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
        const float to = mx > ref[j] + kRefSlack ? mx - kRefBelow : ref[j];
        f[j] = fast_exp2(ref[j] - to);   // 0 from kNoRef
        l[j] *= f[j];
        ref[j] = to;
      }
#pragma unroll
      for (int m = 0; m < C::KM; ++m) {
        acc[m][0] *= f[0];
        acc[m][1] *= f[1];
        acc[m][2] *= f[0];
        acc[m][3] *= f[1];
      }
    }
    // weights, their sums without the scales, and the weights as B
    uint32_t pb[2][C::NP][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[j] = fast_exp2(t[a][2 * i + j] - ref[j]);
          l[j] = fmaf(w[j], inv[a][i], l[j]);
        }
        uint32_t hi = pack_half(w[0], w[1]);
        const float2 hf = unpack_half(hi);
        const uint32_t lo = pack_half(w[0] - hf.x, w[1] - hf.y);
        if constexpr (C::NP == 2) pb[a][1][i] = movmatrix_trans(lo);
        else if (c >= 2) hi = lo;
        pb[a][0][i] = movmatrix_trans(hi);
      }
    // ---- O: k indices 2c, 2c + 1, 2c + 8, 2c + 9 of a half are rows Ra, Rb, Ra + 8, Rb + 8
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      uint32_t v[4][C::VB / 4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = st + ((j & 1) ? vofs_b : vofs_a) + (16 * a + (j >> 1) * 8) * D;
        if constexpr (D == 128) {
          const uint4 x = lds128(at);
          v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
        } else {
          const uint2 x = lds64(at);
          v[j][0] = x.x; v[j][1] = x.y;
        }
      }
#pragma unroll
      for (int k = 0; k < C::VB / 4; ++k) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7362u : 0x5140u;
          uint32_t a0, a1, a2, a3;
          codes_to_half<CODE>(__byte_perm(v[0][k], v[1][k], sel), a0, a1);
          codes_to_half<CODE>(__byte_perm(v[2][k], v[3][k], sel), a2, a3);
          mma_f16(acc[2 * k + half], a0, a1, a2, a3, pb[a][0][0], pb[a][0][1]);
          if constexpr (C::NP == 2) mma_f16(acc[2 * k + half], a0, a1, a2, a3, pb[a][1][0], pb[a][1][1]);
        }
      }
    }
  }

  // ---- the state: this lane's columns' sums complete in every lane
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[j] += __shfl_xor_sync(kFull, l[j], o);
    if (C::kBeside) {
#pragma unroll
      for (int m = 0; m < C::KM; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] += __shfl_xor_sync(kFull, acc[m][i], 2);
    }
  }
  // Dimension of acc[m][2 * i + j]: chunk r, byte 2 m + i of it.
  __device__ __forceinline__ void write_out(int sg) {
    finish();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = column_head(j);
      if (h >= G || (C::kBeside && c >= 2)) continue;
      const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];   // (a NaN stays one)
      T* o = static_cast<T*>(p.out) + ((size_t)sg * G + h) * D + r * C::VB;
#pragma unroll
      for (int m = 0; m < C::KM; ++m) {
        store1(o + 2 * m, acc[m][j] * inv);
        store1(o + 2 * m + 1, acc[m][2 + j] * inv);
      }
    }
  }
  __device__ __forceinline__ void write_state(float* s) {
    finish();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = column_head(j);
      if (h >= G || (C::kBeside && c >= 2)) continue;
      if (r == 0) {
        s[h] = ref[j];
        s[G + h] = l[j];
      }
      float2* o = reinterpret_cast<float2*>(s + 2 * G + h * D + r * C::VB);
#pragma unroll
      for (int m = 0; m < C::KM; ++m) o[m] = make_float2(acc[m][j], acc[m][2 + j]);
    }
  }
};

// What a warp leaves for the CTA's merge.
struct WarpEnd {
  int ended;     // segment that began before the warp and ended in it, or -1
  int open;      // segment still open at the warp's end, or -1
  int began;     // the open segment began in this warp
};

// One merged column over a chain of states.
struct Chain {
  float m, l, a;
  __device__ __forceinline__ void clear() { m = kNoRef; l = 0.f; a = 0.f; }
  __device__ __forceinline__ void add(float m2, float l2, float a2) {
    const float M = fmaxf(m, m2);
    const float f = fast_exp2(m - M), f2 = fast_exp2(m2 - M);
    l = l * f + l2 * f2;
    a = a * f + a2 * f2;
    m = M;
  }
};

// What the ranges are counted in: sequences (dense: the slabs of all their KV
// heads), or the tiles of the segments (hybrid).  The host keeps all slabs of a call
// below 2^31.
// Ranges are equal in units: a slab is one, and the beginning of a segment
// (queries to load, an output to write) kSegCost more before its first slab.
template <bool HYB>
__device__ __forceinline__ int item_slabs(const Q8AttnParams& p, int i, int n_items) {
  if (i >= n_items) return 0;
  if (HYB) return (__ldcg(&p.tile_rows[i]) + kRows - 1) / kRows;
  return (min(max(p.seqlens[i], 0), p.N_max) + kRows - 1) / kRows * p.Hkv;
}
template <bool HYB>
__device__ __forceinline__ int item_units(const Q8AttnParams& p, int slabs) {
  return HYB || slabs == 0 ? slabs : slabs + kSegCost * p.Hkv;
}
// The first slab at or behind unit `rel` of item i, which has `slabs` (rel may lie
// at its end: then the next item's first); `index` gets its number in the item.
template <bool HYB>
__device__ __forceinline__ Start start_at(const Q8AttnParams& p, int slabs, int i, int rel, int& index) {
  if (HYB) {
    const int seg = i / p.ntiles;
    index = rel;
    return Start{seg, i - seg * p.ntiles, rel};
  }
  const int len = slabs / p.Hkv, g = rel / (len + kSegCost), slab = max(rel - g * (len + kSegCost) - kSegCost, 0);
  index = g * len + slab;
  return Start{i * p.Hkv + g, 0, slab};
}

constexpr int kEntries = 2 * kWarps;   // states in a CTA's merge: each warp's ended one, then its open one

template <typename T, int CODE, int D, int G, bool HYB>
__global__ void __launch_bounds__(kThreads, 1) q8_attn_kernel(const __grid_constant__ Q8AttnParams p) {
  using C = Cfg<T, CODE, D, G>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ int s_wsum[kWarps];
  __shared__ int4 s_at[kWarps + 1];     // per warp, and for the range's end: item, its units before, slabs, slabs before
  __shared__ int s_index[kWarps + 1];   // slabs of the call before the warp's first one
  __shared__ WarpEnd s_end[kWarps];
  __shared__ Start s_start[kWarps];
  __shared__ uint32_t s_first, s_valid;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmv)) : "memory");
  }
  pdl_wait();

  // ---- how many slabs there are, and where each warp's begin
  if (blockIdx.x == 0)
    for (int b = tid; b < p.B; b += kThreads) {
      const int n = p.seqlens[b];
      if (n < 0 || n > p.N_max) flag_error(p.err, kErrBadSeqlen);
      if (HYB && p.k_per_seq && n > 0 && p.k_per_seq[b] < 1) flag_error(p.err, kErrBadBudget);
    }
  const int n_items = HYB ? p.B * p.Hkv * p.ntiles : p.B;
  Start s0{0, 0, 0};
  int mine = 0;
  // the ranges of [0, total) units: per CTA, at least one a warp, then per warp
  int c0 = 0, c1 = 0, per_warp = 1;
  auto cut_ranges = [&](int total) {
    const int per_cta = max((int)(((unsigned)total + gridDim.x - 1) / gridDim.x), kWarps);
    c0 = (int)min((long long)total, (long long)per_cta * blockIdx.x);
    c1 = (int)min((long long)total, (long long)c0 + per_cta);
    per_warp = max((c1 - c0 + kWarps - 1) / kWarps, 1);
  };
  // Hands the item to the warps whose ranges begin among its units [lo, lo + units),
  // warp kWarps standing for the end of the CTA's range; `before`: slabs before it.
  auto place = [&](int units, int slabs, int i, int lo, int before) {
    const int hi = lo + units;
    if (units > 0 && hi > c0 && lo <= c1) {
      for (int w = lo > c0 ? (lo - c0 + per_warp - 1) / per_warp : 0; w <= kWarps; ++w) {
        const int u = w < kWarps ? min(c0 + w * per_warp, c1) : c1;
        if (u >= hi) break;
        if (u >= lo) s_at[w] = make_int4(i, lo, slabs, before);
      }
    }
  };
  // (whoever finds no item begins at the call's end)
  auto my_start = [&](int total, int all_slabs) {
    if (tid <= kWarps) {
      const int u = tid < kWarps ? min(c0 + tid * per_warp, c1) : c1;
      if (u >= total) s_at[tid].x = -1;
    }
    __syncthreads();
    if (lane == 0 || (warp == 0 && lane == 1)) {
      const int w = lane == 0 ? warp : kWarps;
      const int u = w < kWarps ? min(c0 + w * per_warp, c1) : c1;
      const int4 at = s_at[w];
      int index = 0;
      Start st{0, 0, 0};
      if (at.x >= 0) st = start_at<HYB>(p, at.z, at.x, u - at.y, index);
      s_index[w] = at.x >= 0 ? at.w + index : all_slabs;
      if (w < kWarps) s_start[w] = st;
    }
    __syncthreads();
    s0 = s_start[warp];
    mine = s_index[warp + 1] - s_index[warp];
  };
  // exclusive prefix of v over the CTA's threads; `sum` gets the total
  auto scan = [&](int v, int& sum) {
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_wsum[warp] = incl;
    __syncthreads();
    int off = 0;
    sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) off += s_wsum[w];
      sum += s_wsum[w];
    }
    return off + incl - v;
  };
  if (p.whole) {
    // segment blockIdx.x is this CTA's
    if ((int)blockIdx.x < p.B * p.Hkv) {
      // (hybrid: it has one tile, its rows below kQ8WholeMax)
      const int rows = HYB ? __ldcg(&p.tile_rows[blockIdx.x]) : min(max(p.seqlens[blockIdx.x / p.Hkv], 0), p.N_max);
      const int total = (rows + kRows - 1) / kRows, per = (total + kWarps - 1) / kWarps, w0 = min(total, per * warp);
      mine = min(total, w0 + per) - w0;
      s0.seg = blockIdx.x;
      s0.slab = w0;
    }
  } else if (n_items <= kThreads) {
    const int slabs = item_slabs<HYB>(p, tid, n_items), units = item_units<HYB>(p, slabs);
    int total, all_slabs;
    const int lo = scan(units, total);
    int before = lo;
    all_slabs = total;
    if (!HYB) {
      __syncthreads();   // the sums were read
      before = scan(slabs, all_slabs);
    }
    cut_ranges(total);
    place(units, slabs, tid, lo, before);
    my_start(total, all_slabs);
  } else {
    int my_units = 0, my_slabs = 0, total, all_slabs;
    for (int i = tid; i < n_items; i += kThreads) {
      const int slabs = item_slabs<HYB>(p, i, n_items);
      my_slabs += slabs;
      my_units += item_units<HYB>(p, slabs);
    }
    scan(my_units, total);
    __syncthreads();     // the sums were read
    scan(my_slabs, all_slabs);
    cut_ranges(total);
    int units_before = 0, slabs_before = 0;
    for (int i0 = 0; i0 < n_items && units_before <= c1; i0 += kThreads) {
      const int slabs = item_slabs<HYB>(p, i0 + tid, n_items), units = item_units<HYB>(p, slabs);
      int round_units, round_slabs;
      __syncthreads();
      const int lo = units_before + scan(units, round_units);
      __syncthreads();
      const int before = slabs_before + scan(slabs, round_slabs);
      place(units, slabs, i0 + tid, lo, before);
      units_before += round_units;
      slabs_before += round_slabs;
    }
    my_start(total, all_slabs);
  }
  if (!HYB) {
    // sequences of no rows give zeros
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
      if (p.seqlens[b] <= 0)
        for (int i = tid; i < p.Hq * D; i += kThreads) store1(static_cast<T*>(p.out) + (size_t)b * p.Hq * D + i, 0.f);
  }
  // ---- the warp's slabs
  const uint32_t ring = smem_u32(smem) + warp * kStages * C::DATA;
  WarpEnd end{-1, -1, 0};
  auto ended_at = [&](int w) {
    return C::kEndedHere ? reinterpret_cast<float*>(smem + C::OFF_ENDED) + w * C::STATE
                         : p.scratch + ((size_t)blockIdx.x * kWarps + w) * C::STATE;
  };
  using Wk = Warp<T, CODE, D, G, HYB>;
  Wk wk(p, ring, smem_u32(smem) + C::OFF_AUX + warp * C::WARP_AUX);
  if (mine > 0) {
    typename Wk::RawQ raw;
    wk.fetch_q(s0.seg, raw);      // (arrives while the first slabs are on their way)
    bool more = wk.begin(s0);
    int copied = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (more && copied < mine) {
        wk.copy(i);
        ++copied;
        more = wk.advance();
      }
    }
    int seg = s0.seg;
    wk.set_q(seg, raw);
    wk.reset();
    bool began = s0.slab == 0 && (!HYB || wk.first_tile(s0.seg, s0.tile));
    int si = 0, so = kStages - 1;     // the stage read next, the stage filled next
    uint32_t phase = 0;
    for (int i = 0; i < copied; ++i) {
      uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_AUX + warp * C::WARP_AUX + kStages * C::AUX) + si;
      // (the warp decides as one: a slab that lands at the very limit must not part its lanes)
      if (!__all_sync(kFull, mbar_wait(bar, phase, p.err, p.wait_ns))) {
        // flagged, and the result is lost; what is still on its way gets as long again
        for (; i < copied; ++i) {
          mbar_wait(bar, phase, p.err, p.wait_ns);
          if (++si == kStages) {
            si = 0;
            phase ^= 1u;
          }
          bar = reinterpret_cast<uint64_t*>(smem + C::OFF_AUX + warp * C::WARP_AUX + kStages * C::AUX) + si;
        }
        break;
      }
      __syncwarp();
      const uint2 hd = lds64(wk.aux + si * C::AUX + C::AUX_HEAD);
      if ((int)hd.x != seg) {
        if (began) wk.write_out(seg);
        else {
          wk.write_state(ended_at(warp));
          end.ended = seg;
        }
        began = true;
        seg = (int)hd.x;
        wk.fetch_q(seg, raw);
        wk.set_q(seg, raw);
        wk.reset();
      }
      if (more && copied < mine) {
        wk.copy(so);
        ++copied;
        more = wk.advance();
      }
      wk.consume(si, hd);
      so = so + 1 == kStages ? 0 : so + 1;
      if (++si == kStages) {
        si = 0;
        phase ^= 1u;
      }
      __syncwarp();   // the stage is free to be written
    }
    // is the last segment complete?  (the cursor stands on the slab after the last)
    const bool done = !p.whole && !(more && wk.seg == seg);
    if (done && began) wk.write_out(seg);
    else {
      // (an open state goes where the warp's ring was)
      wk.write_state(done ? ended_at(warp) : reinterpret_cast<float*>(smem + warp * kStages * C::DATA));
      if (done) end.ended = seg;
      else {
        end.open = seg;
        end.began = began;
      }
    }
  }
  if (lane == 0) s_end[warp] = end;
  __syncthreads();

  float (*s_f)[32] = reinterpret_cast<float (*)[32]>(smem + C::OFF_AUX), (*s_l)[32] = s_f + G, (*s_m)[32] = s_l + G;
  static_assert(3 * G * 32 * 4 <= kWarps * C::WARP_AUX, "factors where the warps' headers were");

  // ---- merge.  Entry 2w is warp w's ended state (of a segment that began before the
  // warp), entry 2w + 1 its open one.  Valid entries of one segment are neighbours:
  // a chain.  A chain's factors first (one warp a head), then its columns.
  if (warp < G) {
    const WarpEnd we = lane < kEntries ? s_end[lane >> 1] : WarpEnd{-1, -1, 0};
    const int h = warp, eseg = lane & 1 ? we.open : we.ended;
    const bool valid = eseg >= 0;
    float m = kNoRef, l = 0.f;
    if (valid) {
      const float* s = lane & 1 ? reinterpret_cast<const float*>(smem + (lane >> 1) * kStages * C::DATA)
                                : ended_at(lane >> 1);
      m = s[h];
      l = s[G + h];
    }
    const uint32_t vmask = __ballot_sync(kFull, valid);
    const uint32_t below = vmask & ((1u << lane) - 1u);
    const int prev = __shfl_sync(kFull, eseg, below ? 31 - __clz(below) : lane);
    const uint32_t firsts = __ballot_sync(kFull, valid && (!below || prev != eseg));
    // the chain's lanes: from its first valid entry up to the next chain's
    const uint32_t upto = firsts & ((2u << lane) - 1u);
    const int c0_lane = upto ? 31 - __clz(upto) : 0;
    const uint32_t after = firsts & ~((2u << lane) - 1u);
    const int c1_lane = after ? __ffs(after) - 2 : 31;
    float M = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(kFull, M, o);
      if (lane - o >= c0_lane) M = fmaxf(M, y);
    }
    M = __shfl_sync(kFull, M, c1_lane);
    const float f = fast_exp2(m - M);
    float L = f * l;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(kFull, L, o);
      if (lane - o >= c0_lane) L += y;
    }
    L = __shfl_sync(kFull, L, c1_lane);
    s_f[h][lane] = valid ? f : 0.f;
    s_m[h][lane] = M;
    s_l[h][lane] = L;
    if (h == 0 && lane == 0) {
      s_valid = vmask;
      s_first = firsts;
    }
  }
  __syncthreads();
  const uint32_t valid = s_valid;
  int part_seg[2] = {-1, -1};
  constexpr int kQuads = G * D / 4;                          // threads a chain takes
  constexpr int kGroups = kThreads / kQuads;                 // chains at once
  uint32_t firsts = s_first;
  for (int chain = 0; firsts; ++chain) {
    const int e0 = __ffs(firsts) - 1;
    firsts &= firsts - 1;
    const uint32_t mine_e = valid & (firsts ? (1u << (__ffs(firsts) - 1)) - 1u : 0xffffffffu) & ~((1u << e0) - 1u);
    const int e1 = 31 - __clz(mine_e);
    const WarpEnd wf = s_end[e0 >> 1];
    const int cseg = e0 & 1 ? wf.open : wf.ended;
    const bool cbegan = (e0 & 1) && wf.began, cended = !(e1 & 1) || p.whole;
    const int slot = cbegan && !cended ? 1 : 0;
    const bool out = cended && (cbegan || p.whole);
    if (!out) part_seg[slot] = cseg;
    if (tid / kQuads != chain % kGroups) continue;
    const int col = (tid % kQuads) * 4, h = col / D, e = col - h * D;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t left = mine_e; left;) {
      float2 x[4], y[4];
      float f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        x[u] = y[u] = make_float2(0.f, 0.f);
        f[u] = 0.f;
        if (left) {
          const int k = __ffs(left) - 1;
          left &= left - 1;
          const float* s = (k & 1 ? reinterpret_cast<const float*>(smem + (k >> 1) * kStages * C::DATA)
                                  : ended_at(k >> 1)) + 2 * G + col;
          f[u] = s_f[h][k];
          x[u] = *reinterpret_cast<const float2*>(s);
          y[u] = *reinterpret_cast<const float2*>(s + 2);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        a.x = fmaf(f[u], x[u].x, a.x);
        a.y = fmaf(f[u], x[u].y, a.y);
        a.z = fmaf(f[u], y[u].x, a.z);
        a.w = fmaf(f[u], y[u].y, a.w);
      }
    }
    const float L = s_l[h][e0];
    if (out) {
      const int b = cseg / p.Hkv, g = cseg - b * p.Hkv;
      const float inv = L == 0.f ? 0.f : 1.f / L;
      store4(static_cast<T*>(p.out) + ((size_t)b * p.Hq + g * G + h) * D + e, a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    } else {
      float* s = p.parts + ((size_t)blockIdx.x * 2 + slot) * C::STATE;
      *reinterpret_cast<float2*>(s + 2 * G + col) = make_float2(a.x, a.y);
      *reinterpret_cast<float2*>(s + 2 * G + col + 2) = make_float2(a.z, a.w);
      if (e == 0) {
        s[h] = s_m[h][e0];
        s[G + h] = L;
      }
    }
  }
  if (tid == 0 && !p.whole) {
    p.part_seg[2 * blockIdx.x] = part_seg[0];
    p.part_seg[2 * blockIdx.x + 1] = part_seg[1];
  }
}

// ---- the states that attention CTAs left open ------------------------------------------
// Grid (attention CTAs, G): block (x, h) merges head h of the segment that CTA x
// left in its slot 1, with the states that later CTAs left of it in slot 0.  A
// thread group of D / 4 lanes takes every kGroups-th state, then the groups'
// states are merged in order.
constexpr int kMergeThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) q8_merge_kernel(const __grid_constant__ Q8AttnParams p) {
  constexpr int LPS = D / 4;                 // lanes a state
  constexpr int kGroups = kMergeThreads / LPS;
  __shared__ float s_acc[kGroups][D], s_m[kGroups], s_l[kGroups];
  pdl_launch_dependents();
  pdl_wait();
  const int first = blockIdx.x, h = blockIdx.y, ctas = gridDim.x, G = gridDim.y;
  const int seg = p.part_seg[2 * first + 1];
  if (seg < 0) return;
  int more = 0;
  for (int i0 = first + 1; i0 < ctas; i0 += kMergeThreads) {
    const int i = i0 + threadIdx.x;
    const int got = __syncthreads_count(i < ctas && p.part_seg[2 * i] == seg);
    more += got;
    if (got < min(kMergeThreads, ctas - i0)) break;
  }
  const int group = threadIdx.x / LPS, col = (threadIdx.x % LPS) * 4;
  const int stride = G * (D + 2);
  Chain ch[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) ch[j].clear();
  for (int i = group; i <= more; i += kGroups) {
    const float* s = p.parts + ((size_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * stride;
    const float m = s[h], l = s[G + h];
    const float2 a = *reinterpret_cast<const float2*>(s + 2 * G + h * D + col);
    const float2 b = *reinterpret_cast<const float2*>(s + 2 * G + h * D + col + 2);
    ch[0].add(m, l, a.x);
    ch[1].add(m, l, a.y);
    ch[2].add(m, l, b.x);
    ch[3].add(m, l, b.y);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s_acc[group][col + j] = ch[j].a;
  if (col == 0) {
    s_m[group] = ch[0].m;
    s_l[group] = ch[0].l;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    Chain t;
    t.clear();
    for (int i = 0; i < kGroups; ++i) t.add(s_m[i], s_l[i], s_acc[i][threadIdx.x]);
    const int b = seg / p.Hkv, g = seg - b * p.Hkv;
    store1(static_cast<T*>(p.out) + ((size_t)b * p.Hq + g * G + h) * D + threadIdx.x, t.l == 0.f ? 0.f : t.a / t.l);
  }
}

// ---- launches ----
int attn_grid(int sms) { return std::min(sms, kQ8MaxCtas); }
// A segment per CTA when that leaves no segment over and none can be longer than
// kQ8WholeMax positions: nothing is left open, and one launch less than splitting.
// The host does not see the lengths, so the rule goes by the table's capacity: short
// sequences in a wide table are split.  (8 KV heads of 128, one sequence that fills its
// table: 512 positions 7.0 us against 10.1 split, 1024 9.4 against 10.2, 2048 14.0 against
// 10.4; eight sequences of 1024: 9.8 against 12.3.)
bool takes_whole(const Q8AttnParams& p, int grid) {
  return (long long)p.B * p.Hkv <= grid && p.N_max <= kQ8WholeMax;
}

// ----------------------------------------------------------------------------------
template <typename T, int CODE, int D, int G, bool HYB>
cudaError_t launch_g(const Q8AttnParams& p, int grid, cudaStream_t st) {
  using C = Cfg<T, CODE, D, G>;
  auto kfn = q8_attn_kernel<T, CODE, D, G, HYB>;
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.run([&] { return cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM); });
  if (e != cudaSuccess) return e;
  return launch_pdl(kfn, dim3(grid), dim3(kThreads), C::SMEM, st, p);
}

template <typename T, int CODE, int D, bool HYB>
cudaError_t launch_h(const Q8AttnParams& p, int grid, cudaStream_t st) {
  switch (p.Hq / p.Hkv) {
    case 1: return launch_g<T, CODE, D, 1, HYB>(p, grid, st);
    case 2: return launch_g<T, CODE, D, 2, HYB>(p, grid, st);
    case 4: return launch_g<T, CODE, D, 4, HYB>(p, grid, st);
    case 8: return launch_g<T, CODE, D, 8, HYB>(p, grid, st);
  }
  return cudaErrorInvalidValue;
}

template <typename T, int CODE, int D>
cudaError_t launch_d(const Q8AttnParams& p, int grid, cudaStream_t st) {
  return p.tile_rows ? launch_h<T, CODE, D, true>(p, grid, st) : launch_h<T, CODE, D, false>(p, grid, st);
}

template <typename T, int CODE>
cudaError_t launch_c(const Q8AttnParams& p, int D, int grid, cudaStream_t st) {
  return D == 128 ? launch_d<T, CODE, 128>(p, grid, st) : launch_d<T, CODE, 64>(p, grid, st);
}

}  // namespace

cudaError_t launch_q8_merge(const Q8AttnParams& p, int dtype, int D, int sms, cudaStream_t st) {
  const int grid = attn_grid(sms);
  if (takes_whole(p, grid)) return cudaSuccess;
  const dim3 g(grid, p.Hq / p.Hkv), b(kMergeThreads);
  cudaError_t e;
  if (dtype == 0)
    e = D == 128 ? launch_pdl(q8_merge_kernel<__nv_bfloat16, 128>, g, b, 0, st, p)
                 : launch_pdl(q8_merge_kernel<__nv_bfloat16, 64>, g, b, 0, st, p);
  else
    e = D == 128 ? launch_pdl(q8_merge_kernel<float, 128>, g, b, 0, st, p)
                 : launch_pdl(q8_merge_kernel<float, 64>, g, b, 0, st, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_q8_attn(const Q8AttnParams& in, int dtype, int code, int D, int sms, cudaStream_t st) {
  const int grid = attn_grid(sms);
  Q8AttnParams p = in;
  p.whole = takes_whole(in, grid);
  cudaError_t e;
  if (dtype == 0)
    e = code == kCodeE4M3 ? launch_c<__nv_bfloat16, kCodeE4M3>(p, D, grid, st)
                          : launch_c<__nv_bfloat16, kCodeInt8>(p, D, grid, st);
  else
    e = code == kCodeE4M3 ? launch_c<float, kCodeE4M3>(p, D, grid, st) : launch_c<float, kCodeInt8>(p, D, grid, st);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace lychee
