// q8_append.cu -- new keys and values into the 8-bit paged cache, rotated on the
// way, and the queries rotated beside them.
//
// Mathematics.  Token i of the m_b new ones of sequence b sits at position p =
// n_b - m_b + i.  Rotation turns dimension pairs (x1, x2), pair j < rot / 2, by
// the table's angle of (p, j): y1 = x1 c - x2 s, y2 = x2 c + x1 s, each product
// and sum rounded once in fp32 (no contraction, so that codes are reproducible
// operation by operation).  Values are not rotated.  The block of a page and head
// takes the scale 2^e of its largest magnitude (q8.cuh); a block that already
// holds rows of the sequence keeps the larger of its old and the new scale, and
// when that grows its old codes are requantised by old / new.  Codes are y / 2^e
// rounded to nearest even; queries are rounded to their type.
//
// Work split.  Every scale has one writer: a CTA takes one (page, head, K or V),
// reads its new rows once into registers, reduces the magnitude and writes codes
// and scale.  No atomics, so results do not depend on scheduling.  Further CTAs
// rotate the queries, a warp taking one token's heads (or a part of them while
// there are few tokens), so that the angles are read once for many heads.  A lane
// takes W dimensions and the W that pair with them, 16 bytes each: 8 of bf16, 4 of
// fp32 (and of bf16 when rot is an odd multiple of 8).  Rows wait as they lie in
// memory and are turned twice, for the magnitude and for the codes: that costs less
// than the registers of their values (64 a thread, 1024 threads an SM).  Bound by
// memory for prompts (8903 tokens of 32 query and 8 KV heads of 128 in bf16: 44 us,
// 4.6 TB/s in and out), by latency for single tokens (2.8 us).
#include <algorithm>

#include "q8.cuh"

namespace lychee {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// W elements as they lie in memory (kept so while they wait: half the registers of
// their fp32 values), and their values.
template <typename T, int W>
struct Raw {
  static constexpr int N = W * (int)sizeof(T) / 4;   // 2, 4 or 8 words
  uint32_t w[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (N == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
      }
    }
  }
  __device__ __forceinline__ void values(float (&o)[W]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 2) {
        const float2 a = bf16x2_to_float2(w[i]);
        o[2 * i] = a.x;
        o[2 * i + 1] = a.y;
      } else {
        o[i] = __uint_as_float(w[i]);
      }
    }
  }
};
template <int W>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&y)[W]) {
  uint32_t w[W / 2];
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&a);
  }
  if constexpr (W == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int W>
__device__ __forceinline__ void store_row(float* p, const float (&y)[W]) {
#pragma unroll
  for (int i = 0; i < W / 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
}
// W values -> W codes at p.
template <int CODE, int W>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&y)[W], float f) {
  const uint32_t lo = quantise4<CODE>(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
  if constexpr (W == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, quantise4<CODE>(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
  else *reinterpret_cast<uint32_t*>(p) = lo;
}

// The 2 W dimensions of lane j of a row: W at a, W at b, and whether they are W
// rotated pairs (pairs W j ...).  Half-split pairs are (i, i + rot / 2); interleaved
// ones (2i, 2i + 1) lie in 2 W consecutive dimensions, as do the dimensions past rot
// (rot is a multiple of 2 W).
struct LaneDims {
  int a, b;
  bool turn;
};
template <int W>
__device__ __forceinline__ LaneDims lane_dims(int j, int rot, bool interleaved) {
  LaneDims l;
  l.turn = 2 * W * j < rot;
  l.a = l.turn && !interleaved ? W * j : 2 * W * j;
  l.b = l.turn && !interleaved ? rot / 2 + W * j : 2 * W * j + W;
  return l;
}

template <int W>
__device__ __forceinline__ void load_angles(const Q8AppendParams& p, int pos, int j, float (&c)[W], float (&s)[W]) {
  const float* at = p.cos_sin + (size_t)pos * p.rot + W * j;
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const float4 x = *(reinterpret_cast<const float4*>(at) + i);
    const float4 y = *(reinterpret_cast<const float4*>(at + p.rot / 2) + i);
    c[4 * i] = x.x; c[4 * i + 1] = x.y; c[4 * i + 2] = x.z; c[4 * i + 3] = x.w;
    s[4 * i] = y.x; s[4 * i + 1] = y.y; s[4 * i + 2] = y.z; s[4 * i + 3] = y.w;
  }
}
template <int W>
__device__ __forceinline__ void turn_pairs(float (&x)[W], float (&y)[W], const float (&c)[W], const float (&s)[W],
                                           bool interleaved) {
  auto turn = [](float& x1, float& x2, float cv, float sv) {
    const float y1 = __fsub_rn(__fmul_rn(x1, cv), __fmul_rn(x2, sv));
    const float y2 = __fadd_rn(__fmul_rn(x2, cv), __fmul_rn(x1, sv));
    x1 = y1;
    x2 = y2;
  };
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < W / 2; ++e) {
      turn(x[2 * e], x[2 * e + 1], c[e], s[e]);
      turn(y[2 * e], y[2 * e + 1], c[W / 2 + e], s[W / 2 + e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) turn(x[e], y[e], c[e], s[e]);
  }
}

// The new tokens of sequence b: [t0, t0 + m) at positions first ...  m = 0 when it
// has none; a sequence whose numbers do not fit is skipped (its `lost` tokens then
// have no position) and flagged.
struct NewRows {
  int t0, m, first, lost;
};
__device__ __forceinline__ NewRows new_rows(const Q8AppendParams& p, int b, bool flag) {
  NewRows r{b, 1, 0, 0};
  const int n = p.seqlens[b];
  bool ok = true;
  if (p.cu_new) {
    r.t0 = p.cu_new[b];
    const int t1 = p.cu_new[b + 1];
    ok = r.t0 >= 0 && t1 >= r.t0 && t1 <= p.T;
    r.m = ok ? t1 - r.t0 : 0;
  } else if (n == 0) {
    r.m = 0;   // an empty place in a padded batch
  }
  if (r.m > 0) {
    const long long cap = (long long)p.c.max_pages << p.c.page_log2;
    ok = n >= r.m && n <= cap && (!p.cos_sin || n <= p.n_pos);
    if (!ok) {
      r.lost = r.m;
      r.m = 0;
    }
  }
  if (!ok && flag) flag_error(p.err, kErrBadSeqlen);
  r.first = n - r.m;
  return r;
}

// The sequence and block of CTA item `blk`: blocks of sequence 0, then of 1, ...
// (with one token a sequence, block b is sequence b's).  Every thread takes part;
// returns the sequence, or -1 past the last block.
__device__ __forceinline__ int find_block(const Q8AppendParams& p, int blk, bool flag, int& j,
                                          NewRows& rows) {
  if (!p.cu_new) {
    rows = new_rows(p, blk, flag);
    j = rows.first >> p.c.page_log2;
    return rows.m > 0 ? blk : -1;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (p.B <= 32) {
    // every warp by itself
    NewRows r{0, 0, 0, 0};
    if (lane < p.B) r = new_rows(p, lane, flag && warp == 0);
    const int first = r.first >> p.c.page_log2;
    const int nb = r.m > 0 ? ((r.first + r.m - 1) >> p.c.page_log2) - first + 1 : 0;
    int incl = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, blk >= incl - nb && blk < incl);
    if (!here) return -1;
    const int l = __ffs(here) - 1;
    j = __shfl_sync(0xffffffffu, first + blk - (incl - nb), l);
    rows.t0 = __shfl_sync(0xffffffffu, r.t0, l);
    rows.m = __shfl_sync(0xffffffffu, r.m, l);
    rows.first = __shfl_sync(0xffffffffu, r.first, l);
    return l;
  }
  __shared__ int s_sum[kWarps], s_b, s_j;
  if (threadIdx.x == 0) s_b = -1;
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    NewRows r{0, 0, 0, 0};
    if (b < p.B) r = new_rows(p, b, flag);
    const int nb = r.m > 0 ? ((r.first + r.m - 1) >> p.c.page_log2) - (r.first >> p.c.page_log2) + 1 : 0;
    int incl = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();   // s_sum of the previous round was read, s_b is set
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += s_sum[w];
      total += s_sum[w];
    }
    const int at = blk - before - (incl - nb);
    if (at >= 0 && at < nb) {
      s_b = b;
      s_j = (r.first >> p.c.page_log2) + at;
    }
    before += total;
    if (before > blk && !flag) break;   // (the flagging CTA looks at every sequence)
  }
  __syncthreads();
  j = s_j;
  const int b = s_b;
  if (b >= 0) rows = new_rows(p, b, false);
  return b;
}

// One (block, head, K or V).  ITERS: rows each lane group may hold.
template <typename T, int CODE, int D, int W, int ITERS>
__device__ __forceinline__ void append_block(const Q8AppendParams& p, int item) {
  constexpr int LPR = D / (2 * W);        // lanes a row
  constexpr int RPI = kThreads / LPR;     // rows at once
  const int units = 2 * p.Hkv;
  const int blk = item / units, u = item % units;
  const int g = u >> 1;
  const bool is_v = u & 1;
  int j = 0;
  NewRows rows{0, 0, 0, 0};
  const int b = find_block(p, blk, u == 0 && (!p.cu_new || blk == 0), j, rows);
  if (b < 0) return;
  const int page_len = 1 << p.c.page_log2, base = j << p.c.page_log2;
  const int lo = max(rows.first, base), hi = min(rows.first + rows.m, base + page_len);
  const int page = p.c.table[(size_t)b * p.c.max_pages + j];
  if (page < 0 || page >= p.c.num_pages) {
    if (threadIdx.x == 0) flag_error(p.err, kErrBadIndex);
    return;
  }
  const size_t unit = (size_t)page * p.Hkv + g;
  uint8_t* codes = const_cast<uint8_t*>(is_v ? p.c.v : p.c.k) + (unit << p.c.page_log2) * D;
  float* scale = const_cast<float*>(is_v ? p.c.v_scale : p.c.k_scale) + unit;
  const bool goes_on = lo > base;         // the block holds rows of the sequence already
  const float old_scale = goes_on ? *scale : 0.f;
  const int l = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  const LaneDims ld = lane_dims<W>(l, is_v || !p.cos_sin ? 0 : p.rot, p.interleaved != 0);
  const long long stride = is_v ? p.v_stride : p.k_stride;
  const T* src = static_cast<const T*>(is_v ? p.v_new : p.k_new) + (size_t)(rows.t0 + lo - rows.first) * stride + g * D;
  Raw<T, W> ra[ITERS], rb[ITERS];
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int r = r0 + i * RPI;
    ra[i].clear();
    rb[i].clear();
    if (lo + r < hi) {
      ra[i].load(src + r * stride + ld.a);
      rb[i].load(src + r * stride + ld.b);
    }
  }
  // the values of row r (turned again for the codes: cheaper than the registers)
  auto row_values = [&](int i, int r, float (&xa)[W], float (&xb)[W]) {
    ra[i].values(xa);
    rb[i].values(xb);
    if (ld.turn) {
      float c[W], s[W];
      load_angles<W>(p, lo + r, l, c, s);
      turn_pairs<W>(xa, xb, c, s, p.interleaved != 0);
    }
  };
  float amax = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int r = r0 + i * RPI;
    if (lo + r < hi) {
      float xa[W], xb[W];
      row_values(i, r, xa, xb);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        // infinities saturate: they do not set the scale
        const float a = fabsf(xa[e]), c = fabsf(xb[e]);
        const bool fa = a < INFINITY, fc = c < INFINITY;
        amax = fmaxf(amax, fmaxf(fa ? a : 0.f, fc ? c : 0.f));
        finite = finite && fa && fc;
      }
    }
  }
  if (!finite) flag_error(p.err, kErrNotFinite);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  __shared__ float s_max[kWarps];
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, s_max[w]);
  const float fresh = exp2_int(scale_exp<CODE>(amax));
  const float now = goes_on ? fmaxf(old_scale, fresh) : fresh;
  if (goes_on && now > old_scale) {
    // the old rows move to the larger scale
    const float ratio = __fdiv_rn(old_scale, now);
    for (int r = r0; r < lo - base; r += RPI) {
      uint2* at = reinterpret_cast<uint2*>(codes + (size_t)r * D + 2 * W * l);
#pragma unroll
      for (int u = 0; u < W / 4; ++u) {
        const uint2 w = at[u];
        const float4 a = codes_to_float<CODE>(w.x), c = codes_to_float<CODE>(w.y);
        at[u] = make_uint2(quantise4<CODE>(a.x * ratio, a.y * ratio, a.z * ratio, a.w * ratio),
                           quantise4<CODE>(c.x * ratio, c.y * ratio, c.z * ratio, c.w * ratio));
      }
    }
  }
  // scales are powers of two: multiplying by the reciprocal divides exactly
  const float inv = __fdiv_rn(1.f, now);
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int r = r0 + i * RPI;
    if (lo + r < hi) {
      uint8_t* dst = codes + (size_t)(lo - base + r) * D;
      float xa[W], xb[W];
      row_values(i, r, xa, xb);
      store_codes<CODE, W>(dst + ld.a, xa, inv);
      store_codes<CODE, W>(dst + ld.b, xb, inv);
    }
  }
  if (threadIdx.x == 0) *scale = now;
}

// A warp: query heads h0 .. h0 + n of one token, its lane groups side by side.
template <typename T, int D, int W>
__device__ __forceinline__ void rotate_q(const Q8AppendParams& p, int cta, int parts) {
  constexpr int LPR = D / (2 * W);
  constexpr int RPW = 32 / LPR;          // heads at once
  constexpr int U = 2;                   // ... and steps in flight (4: fewer warps fit, 52 us against 44)
  const long long item = (long long)cta * kWarps + (threadIdx.x >> 5);
  if (item >= (long long)p.T * parts) return;
  const int t = (int)(item / parts), part = (int)(item - (long long)t * parts);
  const int per = (p.Hq + parts - 1) / parts, h_end = min(p.Hq, (part + 1) * per);
  const int lane = threadIdx.x & 31, l = lane % LPR;
  int b = t;
  if (p.cu_new) {
    if (p.B <= 32) {
      // the last sequence that begins at or before t
      const uint32_t m = __ballot_sync(0xffffffffu, lane < p.B && p.cu_new[min(lane, p.B)] <= t);
      b = m ? 31 - __clz(m) : 0;
    } else {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_new[mid] <= t) lo = mid;
        else hi = mid;
      }
      b = lo;
    }
  }
  const NewRows rows = new_rows(p, b, false);
  if (t < rows.t0 || t >= rows.t0 + rows.m + rows.lost) return;   // behind the last sequence
  const LaneDims ld = lane_dims<W>(l, p.cos_sin ? p.rot : 0, p.interleaved != 0);
  const T* src = static_cast<const T*>(p.q) + (size_t)t * p.q_stride;
  T* dst = static_cast<T*>(p.q_out) + (size_t)t * p.Hq * D;
  if (rows.lost > 0) {
    // no position, no rotated query
    float x[W];
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = NAN;
    for (int h = part * per + lane / LPR; h < h_end; h += RPW) {
      store_row<W>(dst + h * D + ld.a, x);
      store_row<W>(dst + h * D + ld.b, x);
    }
    return;
  }
  float c[W], s[W];
  if (ld.turn) load_angles<W>(p, rows.first + t - rows.t0, l, c, s);
  for (int h0 = part * per + lane / LPR; h0 < h_end; h0 += U * RPW) {
    Raw<T, W> ra[U], rb[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * RPW;
      if (h < h_end) {
        ra[i].load(src + h * D + ld.a);
        rb[i].load(src + h * D + ld.b);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * RPW;
      if (h < h_end) {
        float xa[W], xb[W];
        ra[i].values(xa);
        rb[i].values(xb);
        if (ld.turn) turn_pairs<W>(xa, xb, c, s, p.interleaved != 0);
        store_row<W>(dst + h * D + ld.a, xa);
        store_row<W>(dst + h * D + ld.b, xb);
      }
    }
  }
}

template <typename T, int CODE, int D, int W, int ITERS>
__global__ void __launch_bounds__(kThreads, ITERS > 4 ? 2 : 4) q8_append_kernel(const __grid_constant__ Q8AppendParams p,
                                                             int n_items, int q_parts) {
  pdl_launch_dependents();
  pdl_wait();
  if ((int)blockIdx.x < n_items) append_block<T, CODE, D, W, ITERS>(p, blockIdx.x);
  else rotate_q<T, D, W>(p, (int)blockIdx.x - n_items, q_parts);
}

template <typename T, int CODE, int D, int W>
cudaError_t launch_t(const Q8AppendParams& p, cudaStream_t st) {
  constexpr int LPR = D / (2 * W), RPI = kThreads / LPR, RPW = 32 / LPR;
  const int page = 1 << p.c.page_log2;
  // blocks with new rows: one a sequence, or at most T / page + 2 B (and T)
  long long blocks = p.B;
  if (p.cu_new) blocks = std::min<long long>((long long)p.T / page + 2LL * p.B, p.T);
  const long long items = blocks * 2 * p.Hkv;
  // a warp a token, or fewer heads a warp while the tokens are too few to fill the GPU
  int parts = 1;
  while (parts * RPW < p.Hq && (long long)p.T * parts < 4096) parts *= 2;
  const long long qctas = p.q ? ((long long)p.T * parts + kWarps - 1) / kWarps : 0;
  if (items + qctas == 0) return cudaSuccess;
  if (items + qctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(items + qctas));
  const int need = p.cu_new ? (page + RPI - 1) / RPI : 1;
  cudaError_t e;
  if (need <= 1) e = launch_pdl(q8_append_kernel<T, CODE, D, W, 1>, grid, dim3(kThreads), 0, st, p, (int)items, parts);
  else if (need <= 2) e = launch_pdl(q8_append_kernel<T, CODE, D, W, 2>, grid, dim3(kThreads), 0, st, p, (int)items, parts);
  else if (need <= 4) e = launch_pdl(q8_append_kernel<T, CODE, D, W, 4>, grid, dim3(kThreads), 0, st, p, (int)items, parts);
  else if constexpr (RPI * 4 < 128) e = launch_pdl(q8_append_kernel<T, CODE, D, W, 8>, grid, dim3(kThreads), 0, st, p, (int)items, parts);
  else e = cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <typename T, int CODE>
cudaError_t launch_c(const Q8AppendParams& p, int D, cudaStream_t st) {
  if constexpr (sizeof(T) == 2) {
    if (p.rot % 16 == 0) return D == 128 ? launch_t<T, CODE, 128, 8>(p, st) : launch_t<T, CODE, 64, 8>(p, st);
  }
  return D == 128 ? launch_t<T, CODE, 128, 4>(p, st) : launch_t<T, CODE, 64, 4>(p, st);
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendParams& p, int dtype, int code, int D, cudaStream_t st) {
  if (dtype == 0)
    return code == kCodeE4M3 ? launch_c<__nv_bfloat16, kCodeE4M3>(p, D, st)
                             : launch_c<__nv_bfloat16, kCodeInt8>(p, D, st);
  return code == kCodeE4M3 ? launch_c<float, kCodeE4M3>(p, D, st) : launch_c<float, kCodeInt8>(p, D, st);
}

}  // namespace lychee
