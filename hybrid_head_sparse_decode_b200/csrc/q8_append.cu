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
// rotate the queries.  A row is shared by D / 8 lanes of eight elements each.
// It is bound by memory for prompts and by latency for single tokens.
#include <algorithm>

#include "q8.cuh"

namespace lychee {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsPerItem = 4;   // query heads a lane group turns with one load of the angles

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&o)[4]);
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&o)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
  o[0] = a.x; o[1] = a.y; o[2] = b.x; o[3] = b.y;
}
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&o)[4]) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  o[0] = w.x; o[1] = w.y; o[2] = w.z; o[3] = w.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* y) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, const float* y) {
  *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
}

// The eight dimensions of lane j of a row: four at a, four at b, and whether they
// are four rotated pairs (pairs 4j .. 4j + 3).  Half-split pairs are (i, i + rot /
// 2); interleaved ones (2i, 2i + 1) lie in eight consecutive dimensions, as do the
// dimensions past rot (rot is a multiple of 8).
struct LaneDims {
  int a, b;
  bool turn, adjacent;
};
__device__ __forceinline__ LaneDims lane_dims(int j, int rot, bool interleaved) {
  LaneDims l;
  l.turn = 8 * j < rot;
  l.adjacent = interleaved;
  l.a = l.turn && !interleaved ? 4 * j : 8 * j;
  l.b = l.turn && !interleaved ? rot / 2 + 4 * j : 8 * j + 4;
  return l;
}

__device__ __forceinline__ void turn_pairs(float (&x)[4], float (&y)[4], float4 c, float4 s,
                                           bool adjacent) {
  const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
  auto turn = [](float& x1, float& x2, float cv, float sv) {
    const float y1 = __fsub_rn(__fmul_rn(x1, cv), __fmul_rn(x2, sv));
    const float y2 = __fadd_rn(__fmul_rn(x2, cv), __fmul_rn(x1, sv));
    x1 = y1;
    x2 = y2;
  };
  if (adjacent) {
    turn(x[0], x[1], cc[0], ss[0]);
    turn(x[2], x[3], cc[1], ss[1]);
    turn(y[0], y[1], cc[2], ss[2]);
    turn(y[2], y[3], cc[3], ss[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) turn(x[e], y[e], cc[e], ss[e]);
  }
}

// The new tokens of sequence b: [t0, t0 + m) at positions first ...  m = 0 when it
// has none; a sequence whose numbers do not fit is skipped and flagged.
struct NewRows {
  int t0, m, first;
};
__device__ __forceinline__ NewRows new_rows(const Q8AppendParams& p, int b, bool flag) {
  NewRows r{b, 1, 0};
  const int n = __ldg(&p.seqlens[b]);
  bool ok = true;
  if (p.cu_new) {
    r.t0 = __ldg(&p.cu_new[b]);
    const int t1 = __ldg(&p.cu_new[b + 1]);
    ok = r.t0 >= 0 && t1 >= r.t0 && t1 <= p.T;
    r.m = ok ? t1 - r.t0 : 0;
  } else if (n == 0) {
    r.m = 0;   // an empty place in a padded batch
  }
  if (r.m > 0) {
    const long long cap = (long long)p.c.max_pages << p.c.page_log2;
    ok = n >= r.m && n <= cap && (!p.cos_sin || n <= p.n_pos);
    if (!ok) r.m = 0;
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
  __shared__ int s_sum[kWarps], s_b, s_j;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_b = -1;
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    NewRows r{0, 0, 0};
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
template <typename T, int CODE, int D, int ITERS>
__device__ __forceinline__ void append_block(const Q8AppendParams& p, int item) {
  constexpr int LPR = D / 8;              // lanes a row
  constexpr int RPI = kThreads / LPR;     // rows at once
  const int units = 2 * p.Hkv;
  const int blk = item / units, u = item % units;
  const int g = u >> 1;
  const bool is_v = u & 1;
  int j = 0;
  NewRows rows{0, 0, 0};
  const int b = find_block(p, blk, u == 0 && (!p.cu_new || blk == 0), j, rows);
  if (b < 0) return;
  const int page_len = 1 << p.c.page_log2, base = j << p.c.page_log2;
  const int lo = max(rows.first, base), hi = min(rows.first + rows.m, base + page_len);
  const int page = __ldg(&p.c.table[(size_t)b * p.c.max_pages + j]);
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
  const LaneDims ld = lane_dims(l, is_v || !p.cos_sin ? 0 : p.rot, p.interleaved != 0);
  const T* src = static_cast<const T*>(is_v ? p.v_new : p.k_new) +
                 (size_t)(rows.t0 + lo - rows.first) * (is_v ? p.v_stride : p.k_stride) + g * D;
  const long long stride = is_v ? p.v_stride : p.k_stride;
  float xa[ITERS][4], xb[ITERS][4];
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int r = r0 + i * RPI;
#pragma unroll
    for (int e = 0; e < 4; ++e) xa[i][e] = xb[i][e] = 0.f;
    if (lo + r < hi) {
      load4<T>(src + r * stride + ld.a, xa[i]);
      load4<T>(src + r * stride + ld.b, xb[i]);
    }
  }
  float amax = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int r = r0 + i * RPI;
    if (lo + r < hi) {
      if (ld.turn) {
        const float4* cs = reinterpret_cast<const float4*>(p.cos_sin + (size_t)(lo + r) * p.rot + 4 * l);
        turn_pairs(xa[i], xb[i], __ldg(cs), __ldg(cs + p.rot / 8), ld.adjacent);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // infinities saturate: they do not set the scale
        const float a = fabsf(xa[i][e]), c = fabsf(xb[i][e]);
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
      uint2* at = reinterpret_cast<uint2*>(codes + (size_t)r * D + 8 * l);
      const uint2 w = *at;
      const float4 a = codes_to_float<CODE>(w.x), c = codes_to_float<CODE>(w.y);
      *at = make_uint2(quantise4<CODE>(a.x * ratio, a.y * ratio, a.z * ratio, a.w * ratio),
                       quantise4<CODE>(c.x * ratio, c.y * ratio, c.z * ratio, c.w * ratio));
    }
  }
  // scales are powers of two: multiplying by the reciprocal divides exactly
  const float inv = __fdiv_rn(1.f, now);
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int r = r0 + i * RPI;
    if (lo + r < hi) {
      uint8_t* dst = codes + (size_t)(lo - base + r) * D;
      const float (&a)[4] = xa[i], (&c)[4] = xb[i];
      *reinterpret_cast<uint32_t*>(dst + ld.a) = quantise4<CODE>(
          a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
      *reinterpret_cast<uint32_t*>(dst + ld.b) = quantise4<CODE>(
          c[0] * inv, c[1] * inv, c[2] * inv, c[3] * inv);
    }
  }
  if (threadIdx.x == 0) *scale = now;
}

// kHeadsPerItem query heads of one token per lane group.
template <typename T, int D>
__device__ __forceinline__ void rotate_q(const Q8AppendParams& p, int cta) {
  constexpr int LPR = D / 8;
  constexpr int RPI = kThreads / LPR;
  const int parts = (p.Hq + kHeadsPerItem - 1) / kHeadsPerItem;
  const long long item = (long long)cta * RPI + threadIdx.x / LPR;
  if (item >= (long long)p.T * parts) return;
  const int t = (int)(item / parts), h0 = (int)(item % parts) * kHeadsPerItem;
  const int l = threadIdx.x % LPR;
  int b = t;
  if (p.cu_new) {
    // the last sequence that begins at or before t
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(&p.cu_new[mid]) <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  const NewRows rows = new_rows(p, b, false);
  if (t < rows.t0 || t >= rows.t0 + rows.m) return;   // behind the last sequence, or skipped
  const LaneDims ld = lane_dims(l, p.cos_sin ? p.rot : 0, p.interleaved != 0);
  const T* src = static_cast<const T*>(p.q) + (size_t)t * p.q_stride;
  T* dst = static_cast<T*>(p.q_out) + (size_t)t * p.Hq * D;
  float xa[kHeadsPerItem][4], xb[kHeadsPerItem][4];
#pragma unroll
  for (int i = 0; i < kHeadsPerItem; ++i) {
    if (h0 + i < p.Hq) {
      load4<T>(src + (h0 + i) * D + ld.a, xa[i]);
      load4<T>(src + (h0 + i) * D + ld.b, xb[i]);
    }
  }
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ld.turn) {
    const float4* cs = reinterpret_cast<const float4*>(
        p.cos_sin + (size_t)(rows.first + t - rows.t0) * p.rot + 4 * l);
    c = __ldg(cs);
    s = __ldg(cs + p.rot / 8);
  }
#pragma unroll
  for (int i = 0; i < kHeadsPerItem; ++i) {
    if (h0 + i < p.Hq) {
      if (ld.turn) turn_pairs(xa[i], xb[i], c, s, ld.adjacent);
      store4(dst + (h0 + i) * D + ld.a, xa[i]);
      store4(dst + (h0 + i) * D + ld.b, xb[i]);
    }
  }
}

template <typename T, int CODE, int D, int ITERS>
__global__ void __launch_bounds__(kThreads) q8_append_kernel(const __grid_constant__ Q8AppendParams p,
                                                             int n_items) {
  pdl_launch_dependents();
  pdl_wait();
  if ((int)blockIdx.x < n_items) append_block<T, CODE, D, ITERS>(p, blockIdx.x);
  else rotate_q<T, D>(p, (int)blockIdx.x - n_items);
}

template <typename T, int CODE, int D>
cudaError_t launch_t(const Q8AppendParams& p, cudaStream_t st) {
  constexpr int RPI = kThreads / (D / 8);
  const int page = 1 << p.c.page_log2;
  // blocks with new rows: one a sequence, or at most T / page + 2 B (and T)
  long long blocks = p.B;
  if (p.cu_new) blocks = std::min<long long>((long long)p.T / page + 2LL * p.B, p.T);
  const long long items = blocks * 2 * p.Hkv;
  const int parts = (p.Hq + kHeadsPerItem - 1) / kHeadsPerItem;
  const long long qctas = p.q ? ((long long)p.T * parts + RPI - 1) / RPI : 0;
  if (items + qctas == 0) return cudaSuccess;
  if (items + qctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(items + qctas));
  const int need = p.cu_new ? (page + RPI - 1) / RPI : 1;
  cudaError_t e;
  if (need <= 1) e = launch_pdl(q8_append_kernel<T, CODE, D, 1>, grid, dim3(kThreads), 0, st, p, (int)items);
  else if (need <= 4) e = launch_pdl(q8_append_kernel<T, CODE, D, 4>, grid, dim3(kThreads), 0, st, p, (int)items);
  else e = launch_pdl(q8_append_kernel<T, CODE, D, 8>, grid, dim3(kThreads), 0, st, p, (int)items);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <typename T, int CODE>
cudaError_t launch_c(const Q8AppendParams& p, int D, cudaStream_t st) {
  return D == 128 ? launch_t<T, CODE, 128>(p, st) : launch_t<T, CODE, 64>(p, st);
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendParams& p, int dtype, int code, int D, cudaStream_t st) {
  if (dtype == 0)
    return code == kCodeE4M3 ? launch_c<__nv_bfloat16, kCodeE4M3>(p, D, st)
                             : launch_c<__nv_bfloat16, kCodeInt8>(p, D, st);
  return code == kCodeE4M3 ? launch_c<float, kCodeE4M3>(p, D, st) : launch_c<float, kCodeInt8>(p, D, st);
}

}  // namespace lychee
