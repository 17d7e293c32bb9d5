// q8_sets.cu -- the incoming sets of a hybrid layer over the 8-bit cache, in the
// form its attention reads.
//
// A tile is kQ8Tile positions of one sequence and KV head.  In a group with a
// retrieval head every row below n_b is read, and the sparse heads beside it need
// their sets as bits.  In a group of sparse heads only the union of the sets is
// read: its rows are listed tile by tile as rows of the cache (the page table is
// applied here, once), each with the heads that use it.
//
// One CTA a tile.  A set's entries ascend, so the tile's are found by a search with
// kFan samples a round (39321 entries: two rounds), then set as bits in shared
// memory; the union's words are counted, prefix-summed and expanded.  Every word and
// list entry has one writer.  Further CTAs hand the index rows on (a sparse head's
// set goes on as it came) and check them: an entry out of [0, n_b), not above its
// predecessor or behind the set's end is flagged.  A row that is not a set may be
// missed in part by the search; every access stays in bounds.  Bound by latency:
// dependent loads, and twice the index rows' bytes.
#include <algorithm>

#include "q8.cuh"

namespace lychee {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kWords = kQ8Tile / 32;          // words of a tile's bits
constexpr int kSamples = 4;                   // samples a thread takes in a search
constexpr int kFan = 64 * kSamples;           // ... and a search (two warps) at once
constexpr int kSearches = kThreads / 64;
constexpr int kCopyRow = 16 * kThreads;       // entries a copying CTA takes
// Consecutive entries a thread takes at once (8, 12 and 16 take the same time: sets of 30 % of 131072 positions
// 73.7 us a layer, four sequences up to that 143.3, sets of 45 % and eight heads a group 31.2).
constexpr int kBatch = 8;

// One tile.  The set of sparse head t of the group: entries [from, to) of its row
// lie in the tile.
template <int G>
__device__ __forceinline__ void build_tile(const Q8AttnParams& p, int item) {
  __shared__ uint32_t s_bits[G][kWords];
  __shared__ int s_lo[2 * G], s_hi[2 * G], s_n[kWarps];
  __shared__ int s_sum[kWarps];
  __shared__ uint16_t s_off[kQ8Tile];
  __shared__ uint8_t s_heads[kQ8Tile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = item / p.ntiles, tile = item - seg * p.ntiles;
  const int b = seg / p.Hkv, g = seg - b * p.Hkv;
  const int n = min(max(p.seqlens[b], 0), p.N_max);
  const int base = tile * kQ8Tile, rows = min(max(n - base, 0), kQ8Tile);
  uint32_t sparse = 0;                        // bit t: head t of the group is sparse
#pragma unroll
  for (int t = 0; t < G; ++t) {
    const int h = g * G + t;
    if (!((p.role[h >> 5] >> (h & 31)) & 1u)) sparse |= 1u << t;
  }
  const bool dense = sparse != (1u << G) - 1u;
  if (dense && tid == 0) p.tile_rows[item] = rows;
  if (rows == 0 || sparse == 0) {
    if (!dense && tid == 0) p.tile_rows[item] = 0;
    return;
  }
  const int32_t* row0 = p.idx_in + ((size_t)b * p.Hq + g * G) * p.k;
  for (int i = tid; i < G * kWords; i += kThreads) (&s_bits[0][0])[i] = 0u;
  if (tid < 2 * G) {
    s_lo[tid] = 0;
    s_hi[tid] = p.k;
  }
  __syncthreads();
  // search 2t + e: the first entry of head t's row at or above the tile's begin (e =
  // 0) or end; as unsigned numbers the padding's -1 lies above every position
  for (int s0 = 0; s0 < 2 * G; s0 += kSearches) {
    const int s = s0 + tid / 64, j = tid % 64;
    const bool live = s < 2 * G && ((sparse >> (s >> 1)) & 1u);
    const uint32_t target = (uint32_t)(base + (s & 1) * kQ8Tile);
    const int32_t* row = row0 + (size_t)(s >> 1) * p.k;
    for (int width = p.k; width > 0;) {
      // the answer lies in [lo, hi]: step entries to a sample, the last of each step
      const int step = (width + kFan - 1) / kFan;
      int lo = 0, hi = 0, below = 0;
      if (live) {
        lo = s_lo[s];
        hi = s_hi[s];
        uint32_t v[kSamples];
#pragma unroll
        for (int i = 0; i < kSamples; ++i) {
          const int at = lo + (64 * i + j + 1) * step - 1;
          v[i] = at < hi ? (uint32_t)row[at] : 0xffffffffu;
        }
#pragma unroll
        for (int i = 0; i < kSamples; ++i) below += v[i] < target;
      }
      below = __reduce_add_sync(kFull, below);
      if (lane == 0) s_n[warp] = below;
      __syncthreads();
      if (live && j == 0) {
        // (entries ascend: the samples below the target are the first ones)
        const int c = s_n[warp] + s_n[warp + 1];
        s_lo[s] = min(lo + c * step, hi);
        s_hi[s] = min(lo + (c + 1) * step - 1, hi);
      }
      __syncthreads();
      width = step - 1;
    }
  }
  // the tile's entries as bits, kThreads / G threads a head
  const int per = kThreads / G, t = tid / per;
  if ((sparse >> t) & 1u) {
    const int32_t* row = row0 + (size_t)t * p.k;
    const int to = s_lo[2 * t + 1];
    for (int e0 = s_lo[2 * t] + kBatch * (tid % per); e0 < to; e0 += kBatch * per) {
      int at[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) at[i] = e0 + i < to ? row[e0 + i] - base : -1;
      // neighbours share a word: collect them before the atomic
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const bool in = (unsigned)at[i] < (unsigned)rows;
        if (in) m |= 1u << (at[i] & 31);
        const bool goes_on = in && i + 1 < kBatch && at[(i + 1) % kBatch] >> 5 == at[i] >> 5;
        if (in && !goes_on) {
          atomicOr(&s_bits[t][at[i] >> 5], m);
          m = 0;
        }
      }
    }
  }
  __syncthreads();
  if (dense) {
    for (int i = tid; i < G * kWords; i += kThreads) {
      const int h = i / kWords, w = i % kWords;
      if (((sparse >> h) & 1u) && base / 32 + w < p.nwords)
        p.bitmaps[((size_t)b * p.Hq + g * G + h) * p.nwords + base / 32 + w] = s_bits[h][w];
    }
    return;
  }
  // the union, eight positions a thread
  static_assert(kQ8Tile == 8 * kThreads, "a byte of the bits a thread");
  uint32_t bits[G], u = 0;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    bits[h] = (s_bits[h][tid >> 2] >> (8 * (tid & 3))) & 255u;
    u |= bits[h];
  }
  const int mine = __popc(u);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int at = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) at += s_sum[w];
    total += s_sum[w];
  }
  for (; u; u &= u - 1) {
    const int i = __ffs(u) - 1;
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < G; ++h) m |= ((bits[h] >> i) & 1u) << h;
    s_off[at] = (uint16_t)(8 * tid + i);
    s_heads[at] = (uint8_t)m;
    ++at;
  }
  __syncthreads();
  uint32_t* lr = p.list_rows + (size_t)item * kQ8Tile;
  uint8_t* lh = p.list_heads + (size_t)item * kQ8Tile;
  const int32_t* table = p.c.table + (size_t)b * p.c.max_pages;
#pragma unroll 4
  for (int i = tid; i < total; i += kThreads) {
    const int pos = base + s_off[i], page = table[pos >> p.c.page_log2];
    const bool ok = page >= 0 && page < p.c.num_pages;
    if (!ok) flag_error(p.err, kErrBadIndex);
    // (no page: an absent row that no head uses)
    lr[i] = ok ? ((uint32_t)(page * p.Hkv + g) << p.c.page_log2) + (pos & ((1 << p.c.page_log2) - 1)) : 0xffffffffu;
    lh[i] = ok ? s_heads[i] : 0;
  }
  if (tid == 0) p.tile_rows[item] = total;
}

// kCopyRow entries of one sparse head's index row.
__device__ __forceinline__ void hand_on(const Q8AttnParams& p, int item, int parts) {
  __shared__ uint8_t s_head[kMaxHq];
  if (threadIdx.x == 0) {
    int m = 0;
    for (int h = 0; h < p.Hq; ++h)
      if (!((p.role[h >> 5] >> (h & 31)) & 1u)) s_head[m++] = (uint8_t)h;
  }
  __syncthreads();
  const int pair = item / parts, part = item - pair * parts;
  const int b = pair / p.n_sparse;
  const int n = min(max(p.seqlens[b], 0), p.N_max);
  const size_t row = ((size_t)b * p.Hq + s_head[pair - b * p.n_sparse]) * p.k;
  const int32_t* in = p.idx_in + row;
  constexpr int N = 8;
  const int lane = threadIdx.x & 31;
  bool bad = false;
  const int end = min(p.k, (part + 1) * kCopyRow);
  for (int e0 = part * kCopyRow; e0 < end; e0 += N * kThreads) {
    int v[N], before[N];          // lane 0 also reads the entry before its own
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = e0 + i * kThreads + threadIdx.x;
      v[i] = e < end ? in[e] : -1;
      before[i] = lane == 0 && e > 0 && e < end ? in[e - 1] : -1;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = e0 + i * kThreads + threadIdx.x;
      const int up = __shfl_up_sync(kFull, v[i], 1), prev = lane == 0 ? before[i] : up;
      if (e < end) {
        if (v[i] >= 0) bad = bad || v[i] >= n || (e > 0 && (prev < 0 || v[i] <= prev));
        p.idx_out[row + e] = v[i];
      }
    }
  }
  if (bad) flag_error(p.err, kErrBadIndex);
}

template <int G>
__global__ void __launch_bounds__(kThreads, 3) q8_sets_kernel(const __grid_constant__ Q8AttnParams p, int tiles, int parts,
                                                           int out_words) {
  pdl_launch_dependents();
  pdl_wait();
  uint32_t* out = static_cast<uint32_t*>(p.out);
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < (long long)p.B * p.Hq * out_words;
       i += (long long)gridDim.x * kThreads)
    out[i] = 0u;
  if ((int)blockIdx.x < tiles) build_tile<G>(p, blockIdx.x);
  else hand_on(p, (int)blockIdx.x - tiles, parts);
}

}  // namespace

cudaError_t launch_q8_sets(const Q8AttnParams& p, int dtype, int D, cudaStream_t st) {
  const long long tiles = (long long)p.B * p.Hkv * p.ntiles;
  const int parts = (p.k + kCopyRow - 1) / kCopyRow;
  const long long grid = tiles + (long long)p.B * p.n_sparse * parts;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int out_words = D * (dtype == 0 ? 2 : 4) / 4;
  auto launch = [&](auto kfn) {
    return launch_pdl(kfn, dim3((unsigned)grid), dim3(kThreads), 0, st, p, (int)tiles, parts, out_words);
  };
  cudaError_t e = cudaErrorInvalidValue;
  switch (p.Hq / p.Hkv) {
    case 1: e = launch(q8_sets_kernel<1>); break;
    case 2: e = launch(q8_sets_kernel<2>); break;
    case 4: e = launch(q8_sets_kernel<4>); break;
    case 8: e = launch(q8_sets_kernel<8>); break;
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace lychee
