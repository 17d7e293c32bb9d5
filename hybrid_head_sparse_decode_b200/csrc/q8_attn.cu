// q8_attn.cu -- attention of one query token a sequence over the 8-bit paged
// cache: every position (decode_attn_q8), or a hybrid-head layer whose sparse
// heads read their sets only.
//
// Mathematics.  With c_j, c'_j the codes of key and value j and sk, sv the scales
// of their blocks: s_j = (q . c_j) sk / sqrt(d), p = softmax(s) over every j < n_b
// (or over the head's set), out = sum_j p_j sv c'_j.  A sequence of no rows and an
// empty set give zeros.  Both products run on the tensor cores without a second
// rounding of the cache, and take the scales afterwards.
//   q . c   bf16 queries on e4m3 codes: the codes are an operand as they are, and q
//           is two e4m3 parts, hi = e4m3(q') and lo = e4m3(16 (q' - hi)) with q' = q
//           times a power of two that brings its largest magnitude to [2^7, 2^8): the
//           two hold a bf16 exactly above 2^-13 of the largest, and to 2^-21 of the
//           largest below.  Otherwise codes become halves (exact: both code types
//           fit 11 bits), q' has its largest magnitude in [2^13, 2^14), and fp32
//           queries are held in two halves (22 bits).
//   p . c'  codes become halves.  The weight that multiplies them is w_j = p_j sv_j;
//           it is what must fit a half, so the running reference of the online
//           softmax is the maximum of s_j log2(e) + log2(sv_j), and the normaliser
//           sums w_j / sv_j beside it.  The reference is kept 6 below the maximum
//           seen and moved only when a weight would pass 2^15: weights down to 2^-31
//           of the largest keep a place in the half's range (an 8-bit float's range
//           would lose the many small weights of a long context).  With bf16
//           queries a weight is rounded to 11 bits (the output has 8); with fp32
//           ones it is held in two halves.
//
// Work split.  The unit is a slab of 16 rows of one KV head.  All slabs of the
// call, ordered by sequence, head and position, are cut into one equal range per
// CTA and that into one per warp, whatever the lengths (a sequence's and a head's
// slabs are a segment; a hybrid layer counts only the rows that some head of the
// group uses).  A warp works alone: it brings its slabs into a ring of its own in
// shared memory and runs the G heads of the group over each slab at once; no
// barrier joins the warps before the end.  A full slab is 16 consecutive rows of
// one page: two TMA boxes (K and V).  The rows of a sparse head's set, and a
// slab cut by the sequence's end, come row by row (cp.async, absent rows as
// zeros).  At the end the CTA merges its warps' states of a segment, writes what
// is complete and leaves at most two states open: of a segment that began in an
// earlier CTA and of one that goes on in a later CTA.  The second kernel merges
// those.  When there are fewer segments than CTAs and they are short, every
// segment is one CTA's and nothing is left to merge.  All sums have a fixed order.
//
// Layouts.  Rows lie in shared memory with the TMA's swizzle (16-byte pieces of a
// row XORed with its number).  S = K q^T as m16n8k32 (e4m3) or m16n8k16 (halves)
// with the slab's rows as M: a lane takes 16-byte piece c (c = lane % 4) of its
// two rows; which dimension a k index means is free as long as q agrees, so a
// row's words are, or convert to, A fragments in place.  O^T = V^T P with the
// dimensions as M: a lane takes piece lane / 4 of four rows; interleaving the bytes
// of two rows gives the pairs along k that A wants.  Which row stands at which index
// of M and k is free too: index i is row i ^ 4 (i & 1), which makes both reads
// free of bank conflicts.  P moves from the accumulator layout to B by a
// transpose of 8x8 halves (movmatrix).
#include <algorithm>

#include "q8.cuh"

namespace lychee {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = kQ8Warps;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr float kRefBelow = 6.f;     // the reference lies this far below the maximum (log2)
constexpr float kRefSlack = 15.f;    // and moves when a weight passes it by more than this
constexpr float kNoRef = -1e30f;     // no row yet (finite: differences of two stay numbers)
constexpr uint32_t kFullSlab = 1u << 29;   // stage header: sixteen rows of one page, one scale
constexpr uint32_t kAllHeads = 1u << 30;   // ... and every head uses every row

__device__ __forceinline__ void cp_async16z(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
__device__ __forceinline__ uint32_t lds_u(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_u(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Rows y .. y + 15 of the map's array, all of their bytes, to dst in the map's swizzle.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar),
      "l"(policy)
      : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
               "{%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
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

// Four values -> four e4m3 codes (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
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

template <typename T, int CODE, int D, int G>
struct Cfg {
  static constexpr bool kF8 = sizeof(T) == 2 && CODE == kCodeE4M3;   // q as two e4m3 parts
  static constexpr bool kTwo = sizeof(T) == 4;           // q and the weights in two halves
  static constexpr bool kBeside = kTwo && G <= 4;        // ... in columns 0-3 and 4-7 of one product
  static constexpr int NQ = (kTwo && !kBeside) || kF8 ? 2 : 1;   // products of S per k step
  static constexpr int KQ = kF8 ? D / 32 : D / 16;       // k steps of S
  static constexpr int KM = D / 16;                      // blocks of 16 dimensions of O
  static constexpr int H = D / 64;                       // 16-byte pieces of K a lane takes of a row
  static constexpr int VB = D / 8;                       // bytes of V a lane takes of each of its four rows
  static constexpr int DATA = 32 * D;                    // a stage's rows: K, then V
  static constexpr int OFF_V = 16 * D;
  // beside the rows, per stage: row scales (K; log2 of V's), positions and heads, header
  static constexpr int AUX_S = 0, AUX_META = 128, AUX_HEAD = 192, AUX = 208;
  static constexpr int LIST = kQ8Run * 2;                // a run's rows (hybrid): u16 each
  static constexpr int WARP_AUX = kStages * AUX + LIST + 32;   // and the stages' mbarriers
  static constexpr int OFF_AUX = kWarps * kStages * DATA;
  static constexpr int STATE = G * (D + 2);              // floats of a state: m[G], l[G], acc[G][D]
  static constexpr int SMEM = OFF_AUX + kWarps * WARP_AUX + 1024;   // + alignment slack
  static_assert(WARP_AUX % 16 == 0 && kStages * 8 <= 32, "aligned");
  static_assert(DATA / 2 % 1024 == 0 || D == 64, "swizzled rows on 1024-byte (D = 64: 512-byte) boundaries");
  static_assert(kWarps * STATE * 4 <= OFF_AUX, "the states are merged where the rings were");
};

// Where a range of slabs begins.
struct Start {
  int seg, run, slab;   // segment b * Hkv + g; hybrid: run of the segment, slab of the run
};

// A warp's place in its slabs: the next one to copy.
struct Cursor {
  int seg, b, g, n;
  int at, count;        // dense: slab of the segment, slabs of it.  hybrid: slab of the run, slabs of it
  int run, runs;        // hybrid
  int rows;             // hybrid: rows of the run
  bool packed;          // hybrid: the run's rows are consecutive
  int win;              // dense: the slab that lane 0's table entry belongs to
  int page;             // this lane's table entry of the window / run (-1: not a page)
  float ks, lv;         // ... and the block's scales: K's, log2 of V's
};

template <typename T, int CODE, int D, int G, bool HYB>
struct Warp {
  using C = Cfg<T, CODE, D, G>;
  const Q8AttnParams& p;
  uint32_t ring, aux, list, bars;
  int lane, r, c;
  Cursor cur;
  uint32_t parity;      // bit i: the phase that stage i's mbarrier completes next
  uint32_t gathered;    // bit i: stage i was last filled row by row
  bool mixed;           // hybrid: the cursor's group has a sparse head

  __device__ __forceinline__ Warp(const Q8AttnParams& pp, uint32_t ring_, uint32_t aux_)
      : p(pp), ring(ring_), aux(aux_), list(aux_ + kStages * C::AUX), bars(aux_ + kStages * C::AUX + C::LIST) {
    lane = threadIdx.x & 31;
    r = lane >> 2;
    c = lane & 3;
    parity = gathered = 0;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kStages; ++i)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + 8 * i) : "memory");
      fence_mbar_init();
    }
    __syncwarp();
  }
  __device__ __forceinline__ int length(int b) const { return min(max(__ldg(&p.seqlens[b]), 0), p.N_max); }

  __device__ __forceinline__ bool retrieval(int h) const { return (p.role[h >> 5] >> (h & 31)) & 1u; }
  // This lane's table entry at position `pos` (want: there is one), and its scales.
  __device__ __forceinline__ void load_page(bool want, int pos) {
    cur.page = want ? __ldg(&p.c.table[(size_t)cur.b * p.c.max_pages + (pos >> p.c.page_log2)]) : -1;
    const bool ok = cur.page >= 0 && cur.page < p.c.num_pages;
    if (want && !ok) flag_error(p.err, kErrBadIndex);
    if (!ok) cur.page = -1;
    const int unit = max(cur.page, 0) * p.Hkv + cur.g;
    cur.ks = __ldg(&p.c.k_scale[unit]);
    cur.lv = fast_log2(__ldg(&p.c.v_scale[unit]));
  }

  // ---- the cursor
  __device__ __forceinline__ void enter(int seg) {
    cur.seg = seg;
    cur.b = seg / p.Hkv;
    cur.g = seg - cur.b * p.Hkv;
    cur.n = length(cur.b);
    cur.at = 0;
    cur.win = -64;
    if (HYB) {
      cur.run = 0;
      cur.runs = (cur.n + kQ8Run - 1) / kQ8Run;
      mixed = false;
#pragma unroll
      for (int t = 0; t < G; ++t) mixed = mixed || !retrieval(cur.g * G + t);
    } else {
      cur.count = (cur.n + 15) >> 4;
    }
  }
  // The first run at or after `from` that holds a row (`upto` if none does).
  __device__ __forceinline__ int next_run(int seg, int from, int upto) const {
    const uint8_t* s = p.run_slabs + (size_t)seg * p.runs_stride;
    for (int i0 = from; i0 < upto; i0 += 128) {
      uint32_t k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 32 * j + lane;
        k[j] = i < upto ? __ldcg(s + i) : 0u;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t m = __ballot_sync(kFull, k[j] != 0);
        if (m) return i0 + 32 * j + __ffs(m) - 1;
      }
    }
    return upto;
  }
  // To the first segment after cur.seg that has positions; false if there is none.
  __device__ __forceinline__ bool enter_next() {
    int seg = cur.seg + 1;
    while (seg < p.B * p.Hkv) {
      enter(seg);
      if (cur.n > 0) return true;
      seg = (cur.b + 1) * p.Hkv;
    }
    return false;
  }
  // The rows of run cur.run into the list: entry = position in the run | heads << 8.
  __device__ __forceinline__ void build_run() {
    const int base = cur.run * kQ8Run;
    const int word = lane >> 2, shift = (lane & 3) * 8;   // eight positions a lane
    const int pos0 = base + lane * 8;
    const int left = min(max(cur.n - pos0, 0), 8);
    const uint32_t in = (1u << left) - 1u;
    load_page(lane < (kQ8Run >> p.c.page_log2) && base + (lane << p.c.page_log2) < cur.n,
              base + (lane << p.c.page_log2));
    uint32_t bits[G], u = 0;
#pragma unroll
    for (int t = 0; t < G; ++t) {
      const int h = cur.g * G + t;
      if (retrieval(h)) bits[t] = in;
      else {
        const int w = (base >> 5) + word;
        const uint32_t x = w < p.nwords
                               ? __ldcg(&p.bitmaps[((size_t)cur.b * p.Hq + h) * p.nwords + w]) : 0u;
        bits[t] = (x >> shift) & in;
      }
      u |= bits[t];
    }
    const int mine = __popc(u);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    cur.rows = __shfl_sync(kFull, incl, 31);
    cur.count = (cur.rows + 15) >> 4;
    cur.packed = cur.rows == min(cur.n - base, kQ8Run);
    int slot = incl - mine;
    __syncwarp();   // the previous run's entries were read
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((u >> i) & 1u) {
        uint32_t m = 0;
#pragma unroll
        for (int t = 0; t < G; ++t) m |= ((bits[t] >> i) & 1u) << t;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(list + 2 * slot), "h"((uint16_t)((lane * 8 + i) | (m << 8))) : "memory");
        ++slot;
      }
    }
    __syncwarp();
  }
  __device__ __forceinline__ void begin(const Start& s) {
    enter(s.seg);
    if (HYB) {
      cur.run = s.run;
      build_run();
    }
    cur.at = s.slab;
  }
  // To the next slab.  false: there is none (never, unless lengths or sets change
  // under the call).
  __device__ __forceinline__ bool advance() {
    if (++cur.at < cur.count) return true;
    if (HYB) {
      int run = next_run(cur.seg, cur.run + 1, cur.runs);
      while (run >= cur.runs) {
        if (!enter_next()) return false;
        run = next_run(cur.seg, 0, cur.runs);
      }
      cur.run = run;
      cur.at = 0;
      build_run();
      return true;
    }
    return enter_next();
  }

  // ---- the slab at the cursor into stage `si`
  __device__ __forceinline__ void copy(int si) {
    const uint32_t st = ring + si * C::DATA, ax = aux + si * C::AUX;
    const int log2p = p.c.page_log2, pmask = (1 << log2p) - 1;
    const int i = lane & 15;
    int e_at = 16 * cur.at + i;           // hybrid: this lane's row of the run
    uint32_t myrow = 0, meta;
    bool in;
    float ks, lv;
    if (!HYB || cur.packed) {
      // consecutive positions, all in one page (pages are whole slabs)
      int pos0, wl;
      if (HYB) {
        pos0 = cur.run * kQ8Run + 16 * cur.at;
        wl = (16 * cur.at) >> log2p;
      } else {
        pos0 = 16 * cur.at;
        if ((unsigned)(cur.at - cur.win) >= 32u) {
          cur.win = cur.at;
          load_page(cur.at + lane < cur.count, 16 * (cur.at + lane));
        }
        wl = cur.at - cur.win;
      }
      const int page = __shfl_sync(kFull, cur.page, wl);
      const uint32_t row0 = ((uint32_t)(page * p.Hkv + cur.g) << log2p) + (pos0 & pmask);
      const bool full = page >= 0 && cur.n - pos0 >= 16;
      if (full && lane == 0) {
        const uint32_t bar = bars + 8 * si;
        if ((gathered >> si) & 1u) fence_proxy_async_smem();   // ordinary writes before the TMA's
        asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"((uint32_t)C::DATA)
                     : "memory");
        const uint64_t policy = l2_evict_first_policy();
        tma_rows(st, &p.tmk, (int)row0, bar, policy);
        tma_rows(st + C::OFF_V, &p.tmv, (int)row0, bar, policy);
      }
      ks = __shfl_sync(kFull, cur.ks, wl);
      lv = __shfl_sync(kFull, cur.lv, wl);
      uint32_t heads = 0xffu;
      if (HYB && mixed && e_at < cur.rows) {
        uint16_t e;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(e) : "r"(list + 2 * e_at));
        heads = e >> 8;
      }
      if (full) {
        if (HYB && mixed && lane < 16) sts_u(ax + C::AUX_META + lane * 4, heads << 24);
        if (lane == 0)
          sts128(ax + C::AUX_HEAD, (uint32_t)cur.seg, (uint32_t)pos0 | kFullSlab | (HYB && mixed ? 0u : kAllHeads),
                 __float_as_uint(ks), __float_as_uint(lv));
        gathered &= ~(1u << si);
        return;
      }
      in = page >= 0 && i < cur.n - pos0;
      myrow = row0 + i;
      meta = in ? heads << 24 : 0u;
      if (HYB) meta |= (uint32_t)(pos0 + i);
    } else {
      uint16_t e = 0;
      if (e_at < cur.rows) asm volatile("ld.shared.u16 %0, [%1];" : "=h"(e) : "r"(list + 2 * e_at));
      const int off = e & 255, wl = off >> log2p;
      const int page = __shfl_sync(kFull, cur.page, wl);
      ks = __shfl_sync(kFull, cur.ks, wl);
      lv = __shfl_sync(kFull, cur.lv, wl);
      in = e_at < cur.rows && page >= 0;
      myrow = ((uint32_t)(page * p.Hkv + cur.g) << log2p) + (off & pmask);   // (a run begins on a page)
      meta = in ? (uint32_t)(e >> 8) << 24 : 0u;
    }
    // row by row; lane i (and i + 16) knows row i.  An absent row is zeros with scale 1.
    gathered |= 1u << si;
    if (!in) myrow = 0xffffffffu;
    constexpr int LPR = D / 16, RPI = 32 / LPR;   // lanes a row, rows an instruction
    const int lr = lane / LPR, q = lane % LPR;
#pragma unroll
    for (int j = 0; j < 16 / RPI; ++j) {
      const int R = RPI * j + lr;
      const uint32_t row = __shfl_sync(kFull, myrow, R);
      const bool have = row != 0xffffffffu;
      const size_t at = have ? (size_t)row * D + 16 * q : 0;
      const uint32_t dst = st + R * D + ((D == 128 ? q ^ (R & 7) : q ^ ((R >> 1) & 3)) << 4);
      cp_async16z(dst, p.c.k + at, have ? 16u : 0u);
      cp_async16z(dst + C::OFF_V, p.c.v + at, have ? 16u : 0u);
    }
    sts_u(ax + C::AUX_S + lane * 4, __float_as_uint(!in ? (lane < 16 ? 1.f : 0.f) : lane < 16 ? ks : lv));
    if (lane < 16) sts_u(ax + C::AUX_META + lane * 4, meta);
    if (lane == 0) sts128(ax + C::AUX_HEAD, (uint32_t)cur.seg, 0u, 0u, 0u);
  }

  // ---- the heads' states
  uint32_t qf[C::NQ][C::KQ][2];   // q as B fragments
  float fq[2];                    // powers of two that undo q's scaling, of this lane's two columns
  float ref[2], l[2];             // reference (log2) and sum of p, of this lane's two columns
  float acc[C::KM][4];

  __device__ __forceinline__ int column_head(int j) const { return (C::kBeside ? 2 * (c & 1) : 2 * c) + j; }

  size_t logit_row;               // hybrid: where this lane's first column's logits go
  int logit_cols;                 // ... bit j: column j is a retrieval head (written by this lane)

  struct RawQ {
    float4 x[C::KM];
  };
  __device__ __forceinline__ void fetch_q(int seg, RawQ& raw) const {
    const int b = seg / p.Hkv, g = seg - b * p.Hkv;
    const int t = C::kBeside ? r & 3 : r;
#pragma unroll
    for (int m = 0; m < C::KM; ++m) {
      raw.x[m] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < G)
        raw.x[m] = load_q4<T>(static_cast<const T*>(p.q) + ((size_t)b * p.Hq + g * G + t) * D + (m >> 2) * 64 +
                              16 * c + 4 * (m & 3));
    }
  }
  __device__ __forceinline__ void set_q(int seg, const RawQ& q) {
    if (HYB) {
      const int b = seg / p.Hkv, g = seg - b * p.Hkv;
      logit_row = ((size_t)b * p.Hq + g * G + column_head(0)) * p.N_max;
      logit_cols = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (column_head(j) < G && (!C::kBeside || c < 2) && retrieval(g * G + column_head(j))) logit_cols |= 1 << j;
    }
    const float4 (&x)[C::KM] = q.x;
    float mx = 0.f;
#pragma unroll
    for (int m = 0; m < C::KM; ++m)
      mx = fmaxf(mx, fmaxf(fmaxf(fabsf(x[m].x), fabsf(x[m].y)), fmaxf(fabsf(x[m].z), fabsf(x[m].w))));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    // the largest magnitude to [2^top, 2^(top + 1)) (below 2^-100 the same factor as at 2^-100)
    constexpr int top = C::kF8 ? 7 : 13;
    const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
    const float up = exp2_int(top - e);
    const float down = mx < INFINITY ? exp2_int(e - top) : NAN;   // (an infinite q has no score)
    if constexpr (C::kF8) {
      // x[m] holds four dimensions: two m to a k step of 32
#pragma unroll
      for (int m = 0; m < C::KM; ++m) {
        const float a[4] = {x[m].x * up, x[m].y * up, x[m].z * up, x[m].w * up};
        const uint32_t hi = e4m3x4(a[0], a[1], a[2], a[3]);
        const float4 h = codes_to_float<kCodeE4M3>(hi);
        qf[0][m >> 1][m & 1] = hi;
        qf[C::NQ - 1][m >> 1][m & 1] =
            e4m3x4(16.f * (a[0] - h.x), 16.f * (a[1] - h.y), 16.f * (a[2] - h.z), 16.f * (a[3] - h.w));
      }
    } else {
#pragma unroll
    for (int m = 0; m < C::KM; ++m) {
      const float a = x[m].x * up, bb = x[m].y * up, cc = x[m].z * up, d = x[m].w * up;
      uint32_t w0 = pack_half(a, bb), w1 = pack_half(cc, d);
      if constexpr (C::kTwo) {
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
  __device__ __forceinline__ void consume(int si, uint4 hd, int seg) {
    const uint32_t st = ring + si * C::DATA, ax = aux + si * C::AUX;
    const int R = r ^ ((r & 1) << 2);      // this lane's rows of S: R and R + 8
    // ---- S
    float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t ka = st + R * D + ((D == 128 ? c ^ (R & 7) : c ^ ((R >> 1) & 3)) << 4);
#pragma unroll
    for (int h = 0; h < C::H; ++h) {
      const uint4 lo = lds128(ka ^ (h << 6)), hi = lds128((ka ^ (h << 6)) + 8 * D);
      const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
      if constexpr (C::kF8) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int m = h * 2 + j;
          mma_e4m3(s, wl[2 * j], wh[2 * j], wl[2 * j + 1], wh[2 * j + 1], qf[0][m][0], qf[0][m][1]);
          mma_e4m3(s2, wl[2 * j], wh[2 * j], wl[2 * j + 1], wh[2 * j + 1], qf[C::NQ - 1][m][0], qf[C::NQ - 1][m][1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = h * 4 + j;
          uint32_t a0, a1, a2, a3;
          codes_to_half<CODE>(wl[j], a0, a2);
          codes_to_half<CODE>(wh[j], a1, a3);
          mma_f16((j & 1) ? s2 : s, a0, a1, a2, a3, qf[0][m][0], qf[0][m][1]);
          if constexpr (C::NQ == 2) mma_f16((j & 1) ? s2 : s, a0, a1, a2, a3, qf[C::NQ - 1][m][0], qf[C::NQ - 1][m][1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = C::kF8 ? fmaf(s2[i], 0.0625f, s[i]) : s[i] + s2[i];
    if (C::kBeside) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += __shfl_xor_sync(kFull, s[i], 2);
    }
    // s[0], s[1]: row R, columns 2c and 2c + 1; s[2], s[3]: row R + 8
    const bool full = hd.y & kFullSlab;
    float sk[2] = {__uint_as_float(hd.z), __uint_as_float(hd.z)}, lv[2] = {__uint_as_float(hd.w), __uint_as_float(hd.w)};
    uint32_t meta[2] = {0xff000000u, 0xff000000u};
    if (!full) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sk[i] = lds_f(ax + C::AUX_S + (R + 8 * i) * 4);
        lv[i] = lds_f(ax + C::AUX_S + (16 + R + 8 * i) * 4);
        meta[i] = lds_u(ax + C::AUX_META + (R + 8 * i) * 4);
      }
    } else if (HYB && !(hd.y & kAllHeads)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) meta[i] = lds_u(ax + C::AUX_META + (R + 8 * i) * 4);
    }
    // t: log2 of a row's weight times its scale, -inf where a head does not use it.
    // (Columns beyond the group's heads hold zero queries; nothing reads them.)
    float t[4];
    bool over = false;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float raw = s[2 * i + j] * (sk[i] * fq[j]);
        const int h = column_head(j);
        if (HYB) {
          const bool on = (meta[i] >> (24 + (h & 7))) & 1u;
          if (on && ((logit_cols >> j) & 1)) {
            const int pos = full ? (int)(hd.y & 0xffffffu) + R + 8 * i : (int)(meta[i] & 0xffffffu);
            p.logits[logit_row + (size_t)j * p.N_max + pos] = raw;
          }
          t[2 * i + j] = on ? fmaf(raw, p.scale_log2, lv[i]) : -INFINITY;
        } else {
          t[2 * i + j] = meta[i] ? fmaf(raw, p.scale_log2, lv[i]) : -INFINITY;
        }
        over = over || t[2 * i + j] > ref[j] + kRefSlack;
      }
    if (__any_sync(kFull, over)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = fmaxf(t[j], t[2 + j]);
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
        if (mx > ref[j] + kRefSlack) {
          const float to = mx - kRefBelow;
          const float f = fast_exp2(ref[j] - to);   // 0 from kNoRef
          l[j] *= f;
#pragma unroll
          for (int m = 0; m < C::KM; ++m) {
            acc[m][j] *= f;
            acc[m][2 + j] *= f;
          }
          ref[j] = to;
        }
      }
    }
    // weights, and their sums without the scales
    float w[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float inv = fast_exp2(-lv[i]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        w[2 * i + j] = fast_exp2(t[2 * i + j] - ref[j]);
        l[j] = fmaf(w[2 * i + j], inv, l[j]);
      }
    }
    uint32_t pb[C::kTwo && !C::kBeside ? 2 : 1][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t hi = pack_half(w[2 * i], w[2 * i + 1]);
      if constexpr (C::kTwo) {
        const float2 hf = unpack_half(hi);
        const uint32_t lo = pack_half(w[2 * i] - hf.x, w[2 * i + 1] - hf.y);
        if constexpr (!C::kBeside) pb[1][i] = movmatrix_trans(lo);
        else if (c >= 2) hi = lo;
      }
      pb[0][i] = movmatrix_trans(hi);
    }
    // ---- O: rows Ra, Rb (k indices 2c, 2c + 1), Ra + 8, Rb + 8
    const int Ra = 2 * c, Rb = (2 * c) ^ 5;
    const uint32_t vs = st + C::OFF_V;
    uint32_t v[4][C::VB / 4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int Rv = (j & 1) ? Rb : Ra;
      if constexpr (D == 128) {
        const uint4 x = lds128(vs + Rv * D + ((r ^ (Rv & 7)) << 4) + (j >> 1) * 8 * D);
        v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
      } else {
        const uint2 x = lds64(vs + Rv * D + (((r >> 1) ^ ((Rv >> 1) & 3)) << 4) + (r & 1) * 8 + (j >> 1) * 8 * D);
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
        mma_f16(acc[2 * k + half], a0, a1, a2, a3, pb[0][0], pb[0][1]);
        if constexpr (C::kTwo && !C::kBeside) mma_f16(acc[2 * k + half], a0, a1, a2, a3, pb[1][0], pb[1][1]);
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
  __device__ __forceinline__ void write_out(int seg) {
    finish();
    const int b = seg / p.Hkv, g = seg - b * p.Hkv;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = column_head(j);
      if (h >= G || (C::kBeside && c >= 2)) continue;
      const float inv = l[j] > 0.f ? 1.f / l[j] : 0.f;
      T* o = static_cast<T*>(p.out) + ((size_t)b * p.Hq + g * G + h) * D + r * C::VB;
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
      float* o = s + 2 * G + h * D + r * C::VB;
#pragma unroll
      for (int m = 0; m < C::KM; ++m) {
        o[2 * m] = acc[m][j];
        o[2 * m + 1] = acc[m][2 + j];
      }
    }
  }
};

// What a warp leaves for the CTA's merge.
struct WarpEnd {
  int ended;     // segment that began before the warp and ended in it (its state in global memory), or -1
  int open;      // segment still open at the warp's end (its state in shared memory), or -1
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

__device__ __forceinline__ int warp_sum_int(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// What the ranges are counted in: sequences (dense: the slabs of all their KV
// heads), or sixteen runs (hybrid).
struct Item {
  uint4 runs;           // hybrid: the slab counts, a byte each
  long long slabs;
};
template <bool HYB>
__device__ __forceinline__ Item load_item(const Q8AttnParams& p, int i, int n_items) {
  Item it{make_uint4(0u, 0u, 0u, 0u), 0};
  if (i >= n_items) return it;
  if (HYB) {
    const uint4 x = __ldcg(reinterpret_cast<const uint4*>(p.run_slabs) + i);
    it.runs = x;
    it.slabs = (long long)__dp4a(
        x.x, 0x01010101u, __dp4a(x.y, 0x01010101u, __dp4a(x.z, 0x01010101u, __dp4a(x.w, 0x01010101u, 0u))));
  } else {
    const int n = min(max(__ldg(&p.seqlens[i]), 0), p.N_max);
    it.slabs = (long long)((n + 15) >> 4) * p.Hkv;
  }
  return it;
}
// Slab `rel` of item i.
template <bool HYB>
__device__ __forceinline__ Start start_at(const Q8AttnParams& p, const Item& it, int i, int rel) {
  Start s;
  if (HYB) {
    const uint32_t w[4] = {it.runs.x, it.runs.y, it.runs.z, it.runs.w};
    int at = 0;
    bool found = false;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int k = (int)((w[j >> 2] >> (8 * (j & 3))) & 255u);
      if (!found) {
        if (rel < k) found = true;
        else {
          rel -= k;
          at = min(at + 1, 15);
        }
      }
    }
    const int run = i * 16 + at;
    s.seg = run / p.runs_stride;
    s.run = run - s.seg * p.runs_stride;
    s.slab = rel;
  } else {
    const int len = (int)it.slabs / p.Hkv;
    s.seg = i * p.Hkv + rel / len;
    s.run = 0;
    s.slab = rel % len;
  }
  return s;
}

template <typename T, int CODE, int D, int G, bool HYB>
__global__ void __launch_bounds__(kThreads, 1) q8_attn_kernel(const __grid_constant__ Q8AttnParams p) {
  using C = Cfg<T, CODE, D, G>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ long long s_wsum[kWarps];
  __shared__ Start s_start[kWarps];
  __shared__ WarpEnd s_end[kWarps];
  __shared__ int s_has[kWarps];
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
      const int n = __ldg(&p.seqlens[b]);
      if (n < 0 || n > p.N_max) flag_error(p.err, kErrBadSeqlen);
      if (HYB && p.k_per_seq && n > 0 && __ldg(&p.k_per_seq[b]) < 1) flag_error(p.err, kErrBadBudget);
    }
  const int n_items = HYB ? p.n_run_items : p.B;
  Start s0{0, 0, 0};
  int mine = 0;
  // the ranges of [0, total): per CTA, at least kQ8MinSlabs a warp, then per warp
  long long c0 = 0, c1 = 0, per_warp = 1;
  auto cut_ranges = [&](long long total) {
    const long long per_cta = max((total + gridDim.x - 1) / gridDim.x, (long long)kQ8MinSlabs * kWarps);
    c0 = min(total, per_cta * blockIdx.x);
    c1 = min(total, c0 + per_cta);
    per_warp = max((c1 - c0 + kWarps - 1) / kWarps, 1LL);
    const long long w0 = min(c1, c0 + per_warp * warp);
    mine = (int)(min(c1, w0 + per_warp) - w0);
  };
  // the warps whose ranges begin in [lo, lo + it.slabs)
  auto place = [&](const Item& it, int i, long long lo) {
    const long long hi = lo + it.slabs;
    if (it.slabs > 0 && hi > c0 && lo < c1) {
      int w = lo > c0 ? (int)((lo - c0 + per_warp - 1) / per_warp) : 0;
      for (; w < kWarps && c0 + w * per_warp < min(hi, c1); ++w)
        s_start[w] = start_at<HYB>(p, it, i, (int)(c0 + w * per_warp - lo));
    }
  };
  // exclusive prefix of v over the CTA's threads; `sum` gets the total
  auto scan = [&](long long v, long long& sum) {
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_wsum[warp] = incl;
    __syncthreads();
    long long off = 0;
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
      int k = 0, runs = 0;   // hybrid: this lane's run (there are at most 32), the runs before it
      int total;
      if (HYB) {
        if (lane < p.runs_stride) k = __ldcg(&p.run_slabs[(size_t)blockIdx.x * p.runs_stride + lane]);
        runs = k;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFull, runs, o);
          if (lane >= o) runs += y;
        }
        total = __shfl_sync(kFull, runs, 31);
      } else {
        total = (min(max(__ldg(&p.seqlens[blockIdx.x / p.Hkv]), 0), p.N_max) + 15) >> 4;
      }
      const int per = (total + kWarps - 1) / kWarps, w0 = min(total, per * warp);
      mine = min(total, w0 + per) - w0;
      s0.seg = blockIdx.x;
      s0.slab = w0;
      if (HYB) {
        const uint32_t in = __ballot_sync(kFull, w0 < runs);   // the first lane: the run of slab w0
        s0.run = in ? __ffs(in) - 1 : 0;
        s0.slab = w0 - (__shfl_sync(kFull, runs - k, s0.run));
      }
    }
  } else if (n_items <= kThreads) {
    const Item it = load_item<HYB>(p, tid, n_items);
    long long total;
    const long long lo = scan(it.slabs, total);
    cut_ranges(total);
    place(it, tid, lo);
    __syncthreads();
    s0 = s_start[warp];
  } else {
    long long mine_all = 0, total = 0;
    for (int i = tid; i < n_items; i += kThreads) mine_all += load_item<HYB>(p, i, n_items).slabs;
    scan(mine_all, total);
    cut_ranges(total);
    long long before = 0;
    for (int i0 = 0; i0 < n_items && before < c1; i0 += kThreads) {
      const Item it = load_item<HYB>(p, i0 + tid, n_items);
      __syncthreads();   // the last round's sums were read
      long long round;
      const long long lo = before + scan(it.slabs, round);
      place(it, i0 + tid, lo);
      before += round;
    }
    __syncthreads();
    s0 = s_start[warp];
  }
  if (!HYB) {
    // sequences of no rows give zeros
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
      if (__ldg(&p.seqlens[b]) <= 0)
        for (int i = tid; i < p.Hq * D; i += kThreads) store1(static_cast<T*>(p.out) + (size_t)b * p.Hq * D + i, 0.f);
  }
  // ---- the warp's slabs
  const uint32_t ring = smem_u32(smem) + warp * kStages * C::DATA;
  WarpEnd end{-1, -1, 0};
  float* scratch = p.scratch + ((size_t)blockIdx.x * kWarps + warp) * C::STATE;
  using Wk = Warp<T, CODE, D, G, HYB>;
  Wk wk(p, ring, smem_u32(smem) + C::OFF_AUX + warp * C::WARP_AUX);
  if (mine > 0) {
    typename Wk::RawQ raw;
    wk.fetch_q(s0.seg, raw);      // (arrives while the first slabs are on their way)
    wk.begin(s0);
    // does the first segment begin here?
    bool began = s0.slab == 0;
    if (HYB && began) began = wk.next_run(s0.seg, 0, s0.run) >= s0.run;
    int copied = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (copied > 0 && copied < mine && !wk.advance()) mine = copied;
      if (copied < mine) {
        wk.copy(i);
        ++copied;
      }
      cp_async_commit();
    }
    int seg = s0.seg;
    wk.set_q(seg, raw);
    wk.reset();
    int si = 0, so = kStages - 1;     // the stage read next, the stage filled next
    for (int i = 0; i < mine; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const uint4 hd = lds128(wk.aux + si * C::AUX + C::AUX_HEAD);
      if (hd.y & kFullSlab) {
        uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_AUX + warp * C::WARP_AUX + kStages * C::AUX + C::LIST) + si;
        if (!mbar_wait(bar, (wk.parity >> si) & 1u, p.err)) break;   // (flagged; the result is lost)
        wk.parity ^= 1u << si;
      }
      if ((int)hd.x != seg) {
        if (began) wk.write_out(seg);
        else {
          wk.write_state(scratch);
          end.ended = seg;
        }
        began = true;
        seg = (int)hd.x;
        typename Wk::RawQ raw;
        wk.fetch_q(seg, raw);
        wk.set_q(seg, raw);
        wk.reset();
      }
      if (copied < mine && !wk.advance()) mine = copied;
      if (copied < mine) {
        wk.copy(so);
        ++copied;
      }
      cp_async_commit();
      wk.consume(si, hd, seg);
      si = si + 1 == kStages ? 0 : si + 1;
      so = so + 1 == kStages ? 0 : so + 1;
      __syncwarp();   // the stage is free to be written
    }
    // is the last segment complete?  (the cursor stands on its last copied slab)
    bool last = wk.cur.at + 1 >= wk.cur.count;
    if (HYB && last) last = wk.next_run(seg, wk.cur.run + 1, wk.cur.runs) >= wk.cur.runs;
    if (p.whole) {
      // the CTA merges the segment's states and writes it
      end.open = seg;
      end.began = began;
    } else if (last && began) wk.write_out(seg);
    else if (last) {
      wk.write_state(scratch);
      end.ended = seg;
    } else {
      end.open = seg;
      end.began = began;
    }
  }
  if (lane == 0) {
    s_end[warp] = end;
    s_has[warp] = end.open >= 0;
  }
  __syncthreads();   // every ring is drained
  float* states = reinterpret_cast<float*>(smem);
  if (end.open >= 0) wk.write_state(states + warp * C::STATE);
  __syncthreads();

  // ---- merge: chains of states of one segment across the CTA's warps
  int part_seg[2] = {-1, -1};
  // every warp that has a state has one of the same open segment: the maximum
  // first, then independent terms
  bool single = true;
  int sseg = -1, sbegan = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const WarpEnd we = s_end[w];
    if (we.ended >= 0) single = false;
    if (we.open >= 0) {
      if (sseg >= 0 && we.open != sseg) single = false;
      sseg = we.open;
      sbegan |= we.began;
    }
  }
  if (single) {
    if (sseg >= 0)
      for (int col = tid; col < G * D; col += kThreads) {
        const int h = col / D, e = col - h * D;
        float m[kWarps], l = 0.f, a = 0.f, M = kNoRef;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          m[w] = s_has[w] ? states[w * C::STATE + h] : kNoRef;
          M = fmaxf(M, m[w]);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = fast_exp2(m[w] - M);
          if (s_has[w]) {
            l = fmaf(f, states[w * C::STATE + G + h], l);
            a = fmaf(f, states[w * C::STATE + 2 * G + col], a);
          }
        }
        if (p.whole) {
          const int b = sseg / p.Hkv, g = sseg - b * p.Hkv;
          store1(static_cast<T*>(p.out) + ((size_t)b * p.Hq + g * G + h) * D + e, l > 0.f ? a / l : 0.f);
        } else {
          float* s = p.parts + ((size_t)blockIdx.x * 2 + sbegan) * C::STATE;
          s[2 * G + col] = a;
          if (e == 0) {
            s[h] = M;
            s[G + h] = l;
          }
        }
      }
    part_seg[sbegan] = sseg;
  }
  for (int col = tid; !single && col < G * D; col += kThreads) {
    const int h = col / D, e = col - h * D;
    Chain ch;
    ch.clear();
    int cseg = -1;
    bool cbegan = false;
    auto leave = [&](int slot) {   // an incomplete chain goes to the CTA's slot
      float* s = p.parts + ((size_t)blockIdx.x * 2 + slot) * C::STATE;
      s[2 * G + col] = ch.a;
      if (e == 0) {
        s[h] = ch.m;
        s[G + h] = ch.l;
      }
    };
    part_seg[0] = part_seg[1] = -1;
    for (int w = 0; w < kWarps; ++w) {
      const WarpEnd we = s_end[w];
      if (we.ended >= 0) {
        const float* s = p.scratch + ((size_t)blockIdx.x * kWarps + w) * C::STATE;
        ch.add(s[h], s[G + h], s[2 * G + col]);
        if (cbegan) {
          const int b = we.ended / p.Hkv, g = we.ended - b * p.Hkv;
          store1(static_cast<T*>(p.out) + ((size_t)b * p.Hq + g * G + h) * D + e, ch.l > 0.f ? ch.a / ch.l : 0.f);
        } else {
          leave(0);
          part_seg[0] = we.ended;
        }
        ch.clear();
        cseg = -1;
        cbegan = false;
      }
      if (we.open >= 0) {
        const float* s = states + w * C::STATE;
        if (we.began) cbegan = true;
        cseg = we.open;
        ch.add(s[h], s[G + h], s[2 * G + col]);
      }
    }
    if (cseg >= 0) {
      leave(cbegan ? 1 : 0);
      part_seg[cbegan ? 1 : 0] = cseg;
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
    store1(static_cast<T*>(p.out) + ((size_t)b * p.Hq + g * G + h) * D + threadIdx.x, t.l > 0.f ? t.a / t.l : 0.f);
  }
}

// ---- hybrid: slabs of every run -------------------------------------------------------------
// A run is kQ8Run positions of one segment; its rows are those that some head of
// the group uses: all below n_b in a group with a retrieval head, else the union
// of the sets.  One warp a run.  Also clears the output (segments whose sets are
// all empty have no slab and so no writer).
template <typename T, int D>
__global__ void __launch_bounds__(256) q8_runs_kernel(const __grid_constant__ Q8AttnParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long all = (long long)p.B * p.Hkv * p.runs_stride;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < (long long)p.B * p.Hq * D; i += (long long)gridDim.x * 256)
    store1(static_cast<T*>(p.out) + i, 0.f);
  if (id >= (long long)p.n_run_items * 16) return;
  int rows = 0;
  if (id < all) {
    const int seg = (int)(id / p.runs_stride), run = (int)(id - (long long)seg * p.runs_stride);
    const int b = seg / p.Hkv, g = seg - b * p.Hkv, G = p.Hq / p.Hkv;
    const int n = min(max(__ldg(&p.seqlens[b]), 0), p.N_max);
    const int base = run * kQ8Run, left = min(n - base, kQ8Run);
    bool dense = false;
    for (int t = 0; t < G; ++t) dense = dense || ((p.role[(g * G + t) >> 5] >> ((g * G + t) & 31)) & 1u);
    if (left > 0) {
      if (dense) rows = left;
      else {
        uint32_t u = 0;
        const int w = (base >> 5) + lane;
        if (lane < kQ8Run / 32 && 32 * w < n) {
          for (int t = 0; t < G; ++t) u |= __ldcg(&p.bitmaps[((size_t)b * p.Hq + g * G + t) * p.nwords + w]);
          if (n - 32 * w < 32) u &= (1u << (n - 32 * w)) - 1u;
        }
        rows = warp_sum_int(__popc(u));
      }
    }
  }
  if (lane == 0) p.run_slabs[id] = (uint8_t)((rows + 15) >> 4);
}

// ---- launches ----------------------------------------------------------------------------------
template <typename T, int CODE, int D, int G, bool HYB>
cudaError_t launch_g(const Q8AttnParams& p, int grid, cudaStream_t st) {
  using C = Cfg<T, CODE, D, G>;
  auto kfn = q8_attn_kernel<T, CODE, D, G, HYB>;
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.run([&] { return cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM); });
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(kfn, dim3(grid), dim3(kThreads), C::SMEM, st, p)) != cudaSuccess || p.whole) return e;
  return launch_pdl(q8_merge_kernel<T, D>, dim3(grid, G), dim3(kMergeThreads), 0, st, p);
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
  if (!p.run_slabs) return launch_h<T, CODE, D, false>(p, grid, st);
  const long long runs = (long long)p.n_run_items * 16;
  if ((runs + 7) / 8 > 0x7fffffffLL) return cudaErrorInvalidValue;
  const cudaError_t e = launch_pdl(q8_runs_kernel<T, D>, dim3((unsigned)((runs + 7) / 8)), dim3(256), 0, st, p);
  return e != cudaSuccess ? e : launch_h<T, CODE, D, true>(p, grid, st);
}

template <typename T, int CODE>
cudaError_t launch_c(const Q8AttnParams& p, int D, int grid, cudaStream_t st) {
  return D == 128 ? launch_d<T, CODE, 128>(p, grid, st) : launch_d<T, CODE, 64>(p, grid, st);
}

}  // namespace

cudaError_t launch_q8_attn(const Q8AttnParams& in, int dtype, int code, int D, int sms, cudaStream_t st) {
  const int grid = std::min(sms, kQ8MaxCtas);
  Q8AttnParams p = in;
  // A segment per CTA when that leaves no segment over and none is longer than
  // kQ8WholeMax positions: one launch less than splitting.
  p.whole = (long long)p.B * p.Hkv <= grid && p.N_max <= kQ8WholeMax;
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
