// q8_api.cu -- the C ABI of the 8-bit paged cache (declared in include/lychee.h):
// argument checks, workspace layout and launches.  Host code only; no memory is
// allocated here.
#include <cmath>
#include <cstring>

#include "blocksel.h"
#include "common.cuh"
#include "host.h"
#include "lychee.h"
#include "q8.h"

using namespace lychee;

namespace {

bool pow2_page(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

lychee_status check_q8_shape(const lychee_q8_shape* s) {
  if (!s) return LYCHEE_ERR_INVALID_ARG;
  if (s->B < 1 || s->Hq < 1 || s->Hkv < 1 || s->d < 1 || s->num_pages < 1 || s->max_pages < 1 || s->page < 1)
    return LYCHEE_ERR_INVALID_ARG;
  if (s->dtype != LYCHEE_BF16 && s->dtype != LYCHEE_FP32) return LYCHEE_ERR_INVALID_ARG;
  if (s->code != LYCHEE_E4M3 && s->code != LYCHEE_INT8) return LYCHEE_ERR_INVALID_ARG;
  if (s->Hq % s->Hkv != 0) return LYCHEE_ERR_INVALID_ARG;
  const int G = s->Hq / s->Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return LYCHEE_ERR_UNSUPPORTED;
  if (s->Hq > kMaxHq || (s->d != 64 && s->d != 128) || !pow2_page(s->page)) return LYCHEE_ERR_UNSUPPORTED;
  if ((long long)s->max_pages * s->page > (1 << 24)) return LYCHEE_ERR_UNSUPPORTED;
  // rows are counted in 32 bits
  if ((long long)s->num_pages * s->Hkv * s->page > 0x7fffffffLL) return LYCHEE_ERR_UNSUPPORTED;
  if ((long long)s->B * s->Hq >= (1LL << 24)) return LYCHEE_ERR_UNSUPPORTED;
  // slabs, over all sequences and heads, are counted in 32 bits too
  const long long n_max = (long long)s->max_pages * s->page;
  if ((long long)s->B * s->Hkv * ((n_max + kQ8Tile - 1) / kQ8Tile) * (kQ8Tile / kQ8Slab + 1) > 0x7fffffffLL)
    return LYCHEE_ERR_UNSUPPORTED;
  return LYCHEE_OK;
}

lychee_status check_q8_cache(const lychee_q8_cache* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table) return LYCHEE_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->block_table, 4))
    return LYCHEE_ERR_INVALID_ARG;
  return LYCHEE_OK;
}

Q8Cache cache_of(const lychee_q8_shape* s, const lychee_q8_cache* c) {
  Q8Cache r{};
  r.k = static_cast<const uint8_t*>(c->k);
  r.v = static_cast<const uint8_t*>(c->v);
  r.k_scale = c->k_scale;
  r.v_scale = c->v_scale;
  r.table = c->block_table;
  r.num_pages = s->num_pages;
  r.max_pages = s->max_pages;
  while ((1 << r.page_log2) < s->page) ++r.page_log2;
  return r;
}

int n_max_of(const lychee_q8_shape* s) { return s->max_pages * s->page; }

// Bytes of q, and of out.
size_t rows_bytes(const lychee_q8_shape* s) {
  return (size_t)s->B * s->Hq * s->d * (s->dtype == LYCHEE_BF16 ? 2 : 4);
}

// Workspace: the header with the error word; the states that the attention CTAs
// leave open; for the hybrid step
// (k > 0) also the retrieval heads' logits and the sparse heads' sets as bitmaps
// and row lists.
struct Q8Layout {
  size_t part_seg, parts, scratch, logits, bitmaps, tile_rows, list_rows, list_heads, total;
  int nwords, ntiles;
};
Q8Layout q8_layout(const lychee_q8_shape* s, int k) {
  Q8Layout L{};
  const size_t state = (size_t)(s->Hq / s->Hkv) * (s->d + 2) * 4;
  size_t at = sizeof(WsHeader);
  L.part_seg = at;
  at += align256(kQ8MaxCtas * 2 * sizeof(int32_t));
  L.parts = at;
  at += align256(kQ8MaxCtas * 2 * state);
  L.scratch = at;
  at += align256(kQ8MaxCtas * kQ8Warps * state);
  if (k > 0) {
    const size_t n_max = n_max_of(s);
    L.nwords = (int)((n_max + 31) / 32);
    L.ntiles = (int)((n_max + kQ8Tile - 1) / kQ8Tile);
    const size_t tiles = (size_t)s->B * s->Hkv * L.ntiles;
    L.logits = at;
    at += align256((size_t)s->B * s->Hq * n_max * 4);
    L.bitmaps = at;
    at += align256((size_t)s->B * s->Hq * L.nwords * 4);
    L.tile_rows = at;
    at += align256(tiles * 4);
    L.list_rows = at;
    at += align256(tiles * kQ8Tile * 4);
    L.list_heads = at;
    at += align256(tiles * kQ8Tile);
  }
  L.total = at;
  return L;
}

lychee_status check_sets(const lychee_q8_shape* s, int k, int block) {
  const int n_max = n_max_of(s);
  if (k < 1 || k > n_max || block < 0) return LYCHEE_ERR_INVALID_ARG;
  if (block > 1) {
    if (block % 32 != 0 || block > 1024 || block > k) return LYCHEE_ERR_INVALID_ARG;
    if (block_select_smem(n_max, block) > kBlockSelSmemMax) return LYCHEE_ERR_UNSUPPORTED;
  }
  return LYCHEE_OK;
}

// The codes of a cache as an array of rows of d bytes, in boxes of 32 rows (16 when a
// page has no more)
// whose 16-byte pieces are swizzled over 128 (d = 64: 64) bytes.  False when the
// driver offers no encoder or refuses the map.
bool encode_rows(CUtensorMap* m, const void* base, const lychee_q8_shape* s) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)s->d, (cuuint64_t)s->num_pages * s->Hkv * s->page};
  const cuuint64_t strides[1] = {(cuuint64_t)s->d};
  const cuuint32_t box[2] = {(cuuint32_t)s->d, s->page == 16 ? 16u : 32u};
  const cuuint32_t estr[2] = {1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, s->d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Q8AttnParams attn_params(const lychee_q8_shape* s, const void* q, const lychee_q8_cache* c,
                         const int32_t* seqlens, void* out, uint32_t* err, const Q8Layout& L,
                         void* workspace) {
  Q8AttnParams p{};
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.part_seg = reinterpret_cast<int32_t*>(ws + L.part_seg);
  p.parts = reinterpret_cast<float*>(ws + L.parts);
  p.scratch = reinterpret_cast<float*>(ws + L.scratch);
  p.c = cache_of(s, c);
  p.q = q;
  p.out = out;
  p.seqlens = seqlens;
  p.err = err ? err : &reinterpret_cast<WsHeader*>(ws)->err;
  p.B = s->B; p.Hq = s->Hq; p.Hkv = s->Hkv;
  p.N_max = n_max_of(s);
  p.wait_ns = attn_wait_limit_ns(kWaitLimitNs);
  p.withhold_first = attn_withhold_first_item() ? 1 : 0;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)s->d));
  return p;
}

}  // namespace

extern "C" {

size_t lychee_q8_workspace_size(const lychee_q8_shape* s, int32_t k) {
  if (check_q8_shape(s) != LYCHEE_OK || k < 0 || k > n_max_of(s)) return 0;
  return q8_layout(s, k).total;
}

lychee_status lychee_append_rope_q8(const lychee_q8_shape* s, const lychee_q8_cache* cache,
                                    const lychee_q8_tokens* t, const int32_t* seqlens,
                                    uint32_t* device_error, void* stream) {
  lychee_status st = check_q8_shape(s);
  if (st != LYCHEE_OK) return st;
  if ((st = check_q8_cache(cache)) != LYCHEE_OK) return st;
  if (!t || !t->k || !t->v || !seqlens || t->T < 0) return LYCHEE_ERR_INVALID_ARG;
  if ((t->q != nullptr) != (t->q_out != nullptr)) return LYCHEE_ERR_INVALID_ARG;
  if (!t->cu_new && t->T != s->B) return LYCHEE_ERR_INVALID_ARG;
  const int es = s->dtype == LYCHEE_BF16 ? 2 : 4;
  auto row_ok = [&](const void* p, int64_t stride, int heads) {
    return aligned(p, 16) && stride >= (int64_t)heads * s->d && stride * es % 16 == 0;
  };
  if (!row_ok(t->k, t->k_stride, s->Hkv) || !row_ok(t->v, t->v_stride, s->Hkv)) return LYCHEE_ERR_INVALID_ARG;
  if (t->q && (!row_ok(t->q, t->q_stride, s->Hq) || !aligned(t->q_out, 16))) return LYCHEE_ERR_INVALID_ARG;
  if (t->cos_sin && (t->rot < 8 || t->rot > s->d || t->rot % 8 != 0 || t->n_pos < 1 || !aligned(t->cos_sin, 16)))
    return LYCHEE_ERR_INVALID_ARG;
  if (!aligned(t->cu_new, 4) || !aligned(seqlens, 4) || !aligned(device_error, 4)) return LYCHEE_ERR_INVALID_ARG;
  if (t->q) {
    // rotated queries take the queries' own place or another one
    auto span = [&](int64_t stride, int heads) {
      return t->T > 0 ? ((size_t)(t->T - 1) * stride + (size_t)heads * s->d) * es : 0;
    };
    const size_t out_bytes = (size_t)t->T * s->Hq * s->d * es;
    const bool in_place = t->q_out == t->q && (t->T <= 1 || t->q_stride == (int64_t)s->Hq * s->d);
    if ((!in_place && overlap(t->q_out, out_bytes, t->q, span(t->q_stride, s->Hq))) ||
        overlap(t->q_out, out_bytes, t->k, span(t->k_stride, s->Hkv)) ||
        overlap(t->q_out, out_bytes, t->v, span(t->v_stride, s->Hkv)))
      return LYCHEE_ERR_INVALID_ARG;
  }
  Q8AppendParams p{};
  p.c = cache_of(s, cache);
  p.k_new = t->k;
  p.v_new = t->v;
  p.q = t->q;
  p.q_out = t->q_out;
  p.k_stride = t->k_stride;
  p.v_stride = t->v_stride;
  p.q_stride = t->q_stride;
  p.cos_sin = t->cos_sin;
  p.cu_new = t->cu_new;
  p.seqlens = seqlens;
  p.err = device_error;
  p.B = s->B; p.T = t->T; p.Hq = s->Hq; p.Hkv = s->Hkv;
  p.n_pos = t->n_pos;
  p.rot = t->cos_sin ? t->rot : 0;
  p.interleaved = t->interleaved ? 1 : 0;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      timed(kKindAppend, cs, [&] { return launch_q8_append(p, s->dtype, s->code, s->d, cs); });
  return e == cudaSuccess ? LYCHEE_OK : LYCHEE_ERR_CUDA;
}

lychee_status lychee_decode_attn_q8(const lychee_q8_shape* s, const void* q, const lychee_q8_cache* cache,
                                    const int32_t* seqlens, void* out, void* workspace,
                                    size_t workspace_bytes, uint32_t* device_error, void* stream) {
  lychee_status st = check_q8_shape(s);
  if (st != LYCHEE_OK) return st;
  if ((st = check_q8_cache(cache)) != LYCHEE_OK) return st;
  if (!q || !seqlens || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(seqlens, 4) ||
      !aligned(device_error, 4))
    return LYCHEE_ERR_INVALID_ARG;
  const Q8Layout L = q8_layout(s, 0);
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256))
    return LYCHEE_ERR_WORKSPACE;
  if (overlap(q, rows_bytes(s), out, rows_bytes(s))) return LYCHEE_ERR_INVALID_ARG;
  const int sms = num_sms_current();
  if (sms <= 0) return LYCHEE_ERR_CUDA;
  Q8AttnParams p = attn_params(s, q, cache, seqlens, out, device_error, L, workspace);
  for (int i = 0; i < 4; ++i) p.role[i] = 0xffffffffu;
  if (!encode_rows(&p.tmk, cache->k, s) || !encode_rows(&p.tmv, cache->v, s)) return LYCHEE_ERR_CUDA;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(kKindAttn, cs, [&] { return launch_q8_attn(p, s->dtype, s->code, s->d, sms, cs); });
  if (e == cudaSuccess)
    e = timed(kKindCombine, cs, [&] { return launch_q8_merge(p, s->dtype, s->d, sms, cs); });
  return e == cudaSuccess ? LYCHEE_OK : LYCHEE_ERR_CUDA;
}

lychee_status lychee_hybrid_decode_attn_q8(const lychee_q8_shape* s, int32_t k, int32_t block, const void* q,
                                           const lychee_q8_cache* cache, const int32_t* seqlens,
                                           const int32_t* k_per_seq, const uint8_t* head_role,
                                           const int32_t* idx_in, void* out, int32_t* idx_out,
                                           void* workspace, size_t workspace_bytes, uint32_t* device_error, void* stream) {
  lychee_status st = check_q8_shape(s);
  if (st != LYCHEE_OK) return st;
  if ((st = check_q8_cache(cache)) != LYCHEE_OK) return st;
  if ((st = check_sets(s, k, block)) != LYCHEE_OK) return st;
  int ns = 0;
  if ((st = check_roles(head_role, s->Hq, &ns)) != LYCHEE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int sms = num_sms_current();
  TopkParams tp{};
  tp.B = s->B; tp.Hq = s->Hq; tp.N_max = n_max_of(s); tp.k = k;
  tp.sms = sms;
  tp.empty_ok = 1;
  tp.alone = 1;
  for (int h = 0; h < s->Hq; ++h)
    if (head_role[h] == LYCHEE_ROLE_RETRIEVAL) tp.heads[tp.nheads++] = (uint8_t)h;
  if (ns < s->Hq && block <= 1 && !topk_alone_fits(tp, s->dtype, s->d, cs)) return LYCHEE_ERR_UNSUPPORTED;
  if (!q || !seqlens || !out || !idx_out || (ns > 0 && !idx_in)) return LYCHEE_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(seqlens, 4) || !aligned(k_per_seq, 4) ||
      !aligned(idx_in, 4) || !aligned(idx_out, 4) || !aligned(device_error, 4))
    return LYCHEE_ERR_INVALID_ARG;
  const Q8Layout L = q8_layout(s, k);
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256)) return LYCHEE_ERR_WORKSPACE;
  const size_t sets_bytes = (size_t)s->B * s->Hq * k * sizeof(int32_t);
  if (overlap(q, rows_bytes(s), out, rows_bytes(s)) ||
      (idx_in != idx_out && overlap(idx_in, sets_bytes, idx_out, sets_bytes)))
    return LYCHEE_ERR_INVALID_ARG;
  if (sms <= 0) return LYCHEE_ERR_CUDA;
  Q8AttnParams p = attn_params(s, q, cache, seqlens, out, device_error, L, workspace);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.tile_rows = reinterpret_cast<int32_t*>(ws + L.tile_rows);
  p.list_rows = reinterpret_cast<uint32_t*>(ws + L.list_rows);
  p.list_heads = ws + L.list_heads;
  p.bitmaps = reinterpret_cast<uint32_t*>(ws + L.bitmaps);
  p.logits = reinterpret_cast<float*>(ws + L.logits);
  p.idx_in = idx_in;
  p.idx_out = idx_out;
  p.k_per_seq = k_per_seq;
  p.nwords = L.nwords;
  p.ntiles = L.ntiles;
  p.k = k;
  p.n_sparse = ns;
  fill_roles(p.role, head_role, s->Hq);
  if (!encode_rows(&p.tmk, cache->k, s) || !encode_rows(&p.tmv, cache->v, s)) return LYCHEE_ERR_CUDA;
  if (timed(kKindBuildBits, cs, [&] { return launch_q8_sets(p, s->dtype, s->d, cs); }) != cudaSuccess)
    return LYCHEE_ERR_CUDA;
  if (timed(kKindAttn, cs, [&] { return launch_q8_attn(p, s->dtype, s->code, s->d, sms, cs); }) != cudaSuccess)
    return LYCHEE_ERR_CUDA;
  // (merge and selection need the attention only, but a kernel sees what an earlier one
  // wrote behind its own wait alone, and that is for the kernel before it)
  if (timed(kKindCombine, cs, [&] { return launch_q8_merge(p, s->dtype, s->d, sms, cs); }) != cudaSuccess)
    return LYCHEE_ERR_CUDA;
  if (ns == s->Hq) return LYCHEE_OK;
  // the retrieval heads' selection, as over any cache
  tp.logits = p.logits;
  tp.seqlens = seqlens;
  tp.k_per_seq = k_per_seq;
  tp.idx_out = idx_out;
  tp.err = p.err;
  tp.nwords = L.nwords;
  CombineParams none{};   // B = 0: selection only
  cudaError_t e;
  if (block > 1) {
    BlockSelParams bp{};
    bp.logits = tp.logits;
    bp.seqlens = seqlens;
    bp.k_per_seq = k_per_seq;
    bp.idx_out = idx_out;
    bp.err = tp.err;
    bp.B = tp.B; bp.Hq = tp.Hq; bp.N_max = tp.N_max; bp.nwords = tp.nwords; bp.k = k;
    bp.nheads = tp.nheads;
    bp.block = block;
    bp.empty_ok = 1;
    std::memcpy(bp.heads, tp.heads, sizeof(bp.heads));
    e = timed(kKindTopk, cs, [&] { return launch_block_select_combine(bp, none, s->dtype, s->d, cs); });
  } else {
    e = timed(kKindTopk, cs, [&] { return launch_topk_combine(tp, none, s->dtype, s->d, cs); });
  }
  return e == cudaSuccess ? LYCHEE_OK : LYCHEE_ERR_CUDA;
}

}  // extern "C"
