// q8_attn.cu -- attention of one query token a sequence over the 8-bit paged
// cache.
//
// Mathematics.  s_j = (q . c_j) sk / sqrt(d) with c_j the codes of key j and sk
// the scale of its block; p = softmax(s) over every j < n_b (a head that attends
// to everything) or over the head's set; out = sum_j p_j sv c'_j with the codes
// and scales of the values.  A sequence of no rows and an empty set give zeros.
//
// One CTA per (sequence, query head), one warp per row, an online softmax per
// warp in fp32, the warps' states merged at the end.
#include "q8.cuh"

namespace lychee {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float load1<float>(const float* p) { return *p; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

template <typename T, int CODE, int D>
__global__ void __launch_bounds__(kThreads) q8_attn_kernel(const __grid_constant__ Q8AttnParams p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int E = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_acc[kWarps][D];
  const int bh = blockIdx.x, b = bh / p.Hq, h = bh % p.Hq;
  const int G = p.Hq / p.Hkv, g = h / G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_raw = p.seqlens[b];
  const int n = min(max(n_raw, 0), p.N_max);
  if (threadIdx.x == 0 && h == 0 && n != n_raw) flag_error(p.err, kErrBadSeqlen);
  const bool all = (p.role[h >> 5] >> (h & 31)) & 1u;
  const int32_t* set = p.idx_in + (size_t)bh * p.k;
  const T* q = static_cast<const T*>(p.q) + (size_t)bh * D + lane * E;
  float qr[E], acc[E];
  for (int e = 0; e < E; ++e) {
    qr[e] = load1(q + e);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int rows = all ? n : p.k;
  for (int i = warp; i < rows; i += kWarps) {
    int pos = i;
    if (!all) {
      pos = set[i];
      if (pos < 0) continue;   // past the set's end
      if (pos >= n || (i > 0 && (pos <= set[i - 1] || set[i - 1] < 0))) {
        flag_error(p.err, kErrBadIndex);
        continue;
      }
    }
    const int page = p.c.table[(size_t)b * p.c.max_pages + (pos >> p.c.page_log2)];
    if (page < 0 || page >= p.c.num_pages) {
      flag_error(p.err, kErrBadIndex);
      continue;
    }
    const size_t unit = (size_t)page * p.Hkv + g;
    const size_t row = ((unit << p.c.page_log2) + (pos & ((1 << p.c.page_log2) - 1))) * D;
    float kx[4], vx[4];
    if constexpr (E == 4) {
      const float4 a = codes_to_float<CODE>(*reinterpret_cast<const uint32_t*>(p.c.k + row + lane * E));
      const float4 c = codes_to_float<CODE>(*reinterpret_cast<const uint32_t*>(p.c.v + row + lane * E));
      kx[0] = a.x; kx[1] = a.y; kx[2] = a.z; kx[3] = a.w;
      vx[0] = c.x; vx[1] = c.y; vx[2] = c.z; vx[3] = c.w;
    } else {
      const float4 a = codes_to_float<CODE>(*reinterpret_cast<const uint16_t*>(p.c.k + row + lane * E));
      const float4 c = codes_to_float<CODE>(*reinterpret_cast<const uint16_t*>(p.c.v + row + lane * E));
      kx[0] = a.x; kx[1] = a.y;
      vx[0] = c.x; vx[1] = c.y;
    }
    float dot = 0.f;
    for (int e = 0; e < E; ++e) dot = fmaf(qr[e], kx[e], dot);
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    dot *= p.c.k_scale[unit];
    if (all && p.logits && lane == 0) p.logits[(size_t)bh * p.N_max + pos] = dot;
    const float t = dot * p.scale_log2;
    const float mn = fmaxf(m, t);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn), pr = exp2f(t - mn);
    const float w = pr * p.c.v_scale[unit];
    l = l * a + pr;
    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, vx[e], acc[e] * a);
    m = mn;
  }
  for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float M = -INFINITY, L = 0.f, A = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M);
      L = fmaf(f, s_l[w], L);
      A = fmaf(f, s_acc[w][threadIdx.x], A);
    }
    store1(static_cast<T*>(p.out) + (size_t)bh * D + threadIdx.x, L > 0.f ? A / L : 0.f);
  }
  // a set goes on as it came
  if (p.idx_out) {
    for (int i = threadIdx.x; i < p.k; i += kThreads)
      if (!all) p.idx_out[(size_t)bh * p.k + i] = set[i];
  }
}

template <typename T, int CODE>
cudaError_t launch_c(const Q8AttnParams& p, int D, cudaStream_t st) {
  const dim3 grid((unsigned)(p.B * p.Hq));
  const cudaError_t e = D == 128 ? launch_pdl(q8_attn_kernel<T, CODE, 128>, grid, dim3(kThreads), 0, st, p)
                                 : launch_pdl(q8_attn_kernel<T, CODE, 64>, grid, dim3(kThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q8_attn(const Q8AttnParams& p, int dtype, int code, int D, int sms, cudaStream_t st) {
  if (dtype == 0)
    return code == kCodeE4M3 ? launch_c<__nv_bfloat16, kCodeE4M3>(p, D, st)
                             : launch_c<__nv_bfloat16, kCodeInt8>(p, D, st);
  return code == kCodeE4M3 ? launch_c<float, kCodeE4M3>(p, D, st) : launch_c<float, kCodeInt8>(p, D, st);
}

}  // namespace lychee
