// q8.h -- parameter blocks and launchers of the 8-bit paged cache's kernels (internal).
#pragma once

#include "kernels.h"

namespace lychee {

// The cache of one layer: codes [num_pages, Hkv, page, D] of 8 bits, one fp32
// scale per page and head, and the pages of each sequence.
struct Q8Cache {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;      // [num_pages, Hkv]
  const float* v_scale;
  const int32_t* table;      // [B, max_pages]: page of positions [j * page, (j + 1) * page)
  int num_pages, max_pages;
  int page_log2;             // page = 1 << page_log2 positions (16 .. 128)
};

// New rows into the cache, rotated and quantised; queries rotated (q8_append.cu).
struct Q8AppendParams {
  Q8Cache c;                 // written: k, v, k_scale, v_scale
  const void* k_new;         // [T, Hkv, D], rows of one token k_stride elements apart
  const void* v_new;
  const void* q;             // [T, Hq, D] or null
  void* q_out;               // [T, Hq, D]
  long long k_stride, v_stride, q_stride;   // elements from one token to the next
  const float* cos_sin;      // [n_pos, rot]: cosines, then sines; null: no rotation
  const int32_t* cu_new;     // [B + 1] or null: one token a sequence
  const int32_t* seqlens;    // [B], the new tokens included
  uint32_t* err;             // or null
  int B, T, Hq, Hkv, n_pos, rot, interleaved;
};
cudaError_t launch_q8_append(const Q8AppendParams& p, int dtype, int code, int D, cudaStream_t st);

// Attention of one query token a sequence over the cache (q8_attn.cu).
constexpr int kQ8Warps = 12;       // warps of an attention CTA (one CTA an SM)
constexpr int kQ8Stages = 2;       // slabs in a warp's ring
constexpr int kQ8Slab = 32;        // rows of a slab
constexpr int kQ8MaxCtas = 160;    // attention CTAs at most (the workspace holds that many states)
constexpr int kQ8WholeMax = 1024;  // positions of the widest table whose segments are one CTA's each
constexpr int kQ8Tile = 4096;      // positions of a tile (hybrid: the unit whose rows are listed)
struct Q8AttnParams {
  Q8Cache c;
  const void* q;             // [B, Hq, D]
  void* out;                 // [B, Hq, D]
  const int32_t* seqlens;    // [B]
  uint32_t* err;             // the caller's word, or the workspace's
  float* parts;              // [CTAs, 2, G * (D + 2)]: states a CTA left open: of a segment that
                             // began before it, of one that began in it; m[G], l[G], acc[G][D]
  int32_t* part_seg;         // [CTAs, 2]: their segments (sequence * Hkv + KV head), -1: none
  float* scratch;            // [CTAs, kQ8Warps, G * (D + 2)]: a state a warp ended on its way
  int B, Hq, Hkv, N_max;
  float scale_log2;          // log2(e) / sqrt(D)
  uint32_t role[4];          // bit h set: head h attends to every position
  // hybrid layer only (tile_rows null: every head attends to every position)
  int32_t* tile_rows;        // [B * Hkv, ntiles]: rows of each tile that some head of the group uses
  uint32_t* list_rows;       // [B * Hkv, ntiles, kQ8Tile]: in groups of sparse heads those rows (of the cache)
  uint8_t* list_heads;       // ... and the heads of the group that use each
  uint32_t* bitmaps;         // [B, Hq, nwords]: the sets of sparse heads beside a retrieval head
  float* logits;             // [B, Hq, N_max]: raw q.k of the retrieval heads
  const int32_t* idx_in;     // [B, Hq, k]: sets of the sparse heads
  int32_t* idx_out;          // [B, Hq, k]: they go on as they came
  const int32_t* k_per_seq;  // [B] or null (checked here)
  int nwords, ntiles, k, n_sparse;
  unsigned long long wait_ns;   // how long a wait for a slab may take
  int withhold_first;        // test only: a warp's first stage expects an arrival that never comes
  int whole;                 // 1: CTA x takes segment x whole, nothing is left open
  // the cache's codes as rows of D bytes, boxes of 32 rows (pages of 16: 16 rows), swizzled by D bytes
  alignas(64) CUtensorMap tmk;
  alignas(64) CUtensorMap tmv;
};
// The sparse heads' sets as tile_rows, list_* and bitmaps, their rows to idx_out, and
// zeros to out (segments without rows have no other writer) (q8_sets.cu).
cudaError_t launch_q8_sets(const Q8AttnParams& p, int dtype, int D, cudaStream_t st);
cudaError_t launch_q8_attn(const Q8AttnParams& p, int dtype, int code, int D, int sms,
                           cudaStream_t st);
// The states it left open.
cudaError_t launch_q8_merge(const Q8AttnParams& p, int dtype, int D, int sms, cudaStream_t st);

}  // namespace lychee
