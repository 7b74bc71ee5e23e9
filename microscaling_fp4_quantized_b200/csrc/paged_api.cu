// C ABI of the paged cache (declared in include/sage_fp4.h): argument checks and launches.
// Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "paged.h"
#include "sage_fp4.h"

namespace {

constexpr int kMaxPageSize = 65536;

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_dtype(int d) { return d == SAGE_BF16 || d == SAGE_F16; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

bool valid_stride(int64_t s, int unit) { return s >= 0 && s % unit == 0 && s < (int64_t(1) << 40); }

// Strides of rows that are written: two rows of one tensor must not overlap.
bool apart(int64_t stride, int64_t count, int D) { return count <= 1 || stride >= D; }

sage_status_t check_cache(const sage_fp4_cache_t* c) {
  if (c == nullptr) return SAGE_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return SAGE_ERR_UNSUPPORTED;
  if (!valid_dtype(c->dtype)) return SAGE_ERR_INVALID_ARG;
  if (c->format != SAGE_CACHE_16BIT && c->format != SAGE_CACHE_FP4) return SAGE_ERR_INVALID_ARG;
  const bool fp4 = c->format == SAGE_CACHE_FP4;
  if (c->num_pages < 0 || c->page_size < 1 || c->Hkv < 1) return SAGE_ERR_INVALID_ARG;
  if (c->page_size > kMaxPageSize || c->Hkv > 65535) return SAGE_ERR_UNSUPPORTED;
  for (const int64_t* s : {c->k_stride, c->v_stride}) {
    const int64_t counts[3] = {c->num_pages, c->Hkv, c->page_size};
    __int128 last = 0;
    for (int i = 0; i < 3; ++i) {
      if (!valid_stride(s[i], fp4 ? c->D : 8) || !apart(s[i], counts[i], c->D)) return SAGE_ERR_INVALID_ARG;
      last += static_cast<__int128>(std::max<int64_t>(counts[i] - 1, 0)) * s[i];
    }
    // The decode kernel holds row offsets in 32-bit units of 16 bytes (all ones: no row).
    if (last / (fp4 ? 32 : 8) >= 0xffffffff) return SAGE_ERR_UNSUPPORTED;
  }
  if (c->num_pages > 0) {
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SAGE_ERR_INVALID_ARG;
    if (fp4 && (!aligned(c->k_sf, 8) || !aligned(c->v_sf, 8))) return SAGE_ERR_INVALID_ARG;
  }
  return SAGE_OK;
}

sage_status_t check_batch(const sage_fp4_cache_t* c, const sage_fp4_batch_t* b, bool rows, int total) {
  if (b == nullptr || b->B < 0 || b->table_width < 0 || b->table_stride < 0 || total < 0) return SAGE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(b->table_width) * c->page_size > (int64_t(1) << 30)) return SAGE_ERR_UNSUPPORTED;
  if (b->B == 0) return SAGE_OK;
  if (!aligned(b->seq_lens, 4) || (b->table_width > 0 && !aligned(b->page_table, 4))) return SAGE_ERR_INVALID_ARG;
  if (rows) {
    if (b->cu_seqlens == nullptr ? total != b->B : !aligned(b->cu_seqlens, 4)) return SAGE_ERR_INVALID_ARG;
  }
  return SAGE_OK;
}

sage_status_t check_rope(const sage_fp4_rope_t* r, int D) {
  if (r == nullptr) return SAGE_OK;
  if (!std::isfinite(r->eps) || r->eps < 0.0f) return SAGE_ERR_INVALID_ARG;
  for (const void* w : {r->q_weight, r->k_weight})
    if (w != nullptr && !aligned(w, 16)) return SAGE_ERR_INVALID_ARG;
  if (r->rope == nullptr) return SAGE_OK;
  if (!aligned(r->rope, 16) || r->rope_len < 0) return SAGE_ERR_INVALID_ARG;
  if (r->rotary_dim <= 0 || r->rotary_dim > D || r->rotary_dim % 32 != 0) return SAGE_ERR_UNSUPPORTED;
  return SAGE_OK;
}

// counts: how many of (sequence, head, token) the rows have.
sage_status_t check_rows(const sage_fp4_rows_t* r, int64_t B, int64_t N, int D) {
  if (r == nullptr || r->heads == 0) return SAGE_OK;
  if (r->heads < 0) return SAGE_ERR_INVALID_ARG;
  if (r->heads > 65535) return SAGE_ERR_UNSUPPORTED;
  if (!aligned(r->x, 16) || !aligned(r->y, 16)) return SAGE_ERR_INVALID_ARG;
  const int64_t counts[3] = {B, r->heads, N};
  for (int i = 0; i < 3; ++i) {
    if (!valid_stride(r->x_stride[i], 8) || !valid_stride(r->y_stride[i], 8)) return SAGE_ERR_INVALID_ARG;
    if (!apart(r->y_stride[i], counts[i], D)) return SAGE_ERR_INVALID_ARG;
    if (r->x == r->y && counts[i] > 1 && r->x_stride[i] != r->y_stride[i]) return SAGE_ERR_INVALID_ARG;
  }
  return SAGE_OK;
}

sage::Strides strides(const int64_t s[3]) { return sage::Strides{s[0], s[1], s[2]}; }

sage::CacheView view_of(const sage_fp4_cache_t& c, const sage_fp4_batch_t& b) {
  sage::CacheView v;
  std::memset(&v, 0, sizeof(v));
  v.k = c.k;
  v.v = c.v;
  v.k_sf = c.k_sf;
  v.v_sf = c.v_sf;
  v.sk = strides(c.k_stride);
  v.sv = strides(c.v_stride);
  v.num_pages = c.num_pages;
  v.Hkv = c.Hkv;
  v.page = sage::fast_div(static_cast<uint32_t>(c.page_size));
  v.table = b.page_table;
  v.table_stride = b.table_stride;
  v.capacity = b.table_width * c.page_size;
  v.lens = b.seq_lens;
  v.cu = b.cu_seqlens;
  v.B = b.B;
  return v;
}

void set_rope(sage::RowsParams* p, const sage_fp4_rope_t* r) {
  if (r == nullptr) return;
  p->qw = r->q_weight;
  p->kw = r->k_weight;
  p->w32 = r->weight_f32 ? 1 : 0;
  p->eps = r->eps;
  p->rope = r->rope;
  p->rope_len = r->rope != nullptr ? r->rope_len : 0;
  p->R = r->rope != nullptr ? r->rotary_dim : 0;
  p->interleaved = r->interleaved ? 1 : 0;
}

void set_q(sage::RowsParams* p, const sage_fp4_rows_t* q) {
  if (q == nullptr || q->heads == 0) return;
  p->Hq = q->heads;
  p->q = q->x;
  p->qo = q->y;
  p->sq = strides(q->x_stride);
  p->sqo = strides(q->y_stride);
}

// The decode problem's split of the query heads, its grid bound and its workspace.
struct DecodePlan {
  int group, chunks, chunk_heads, NT, max_grid;
  size_t rec, ml, o, bytes;
};

sage_status_t plan_decode(const sage_fp4_cache_t* c, const sage_fp4_batch_t* b, int Hq, DecodePlan* d) {
  if (sage_status_t s = check_cache(c); s != SAGE_OK) return s;
  if (sage_status_t s = check_batch(c, b, false, 0); s != SAGE_OK) return s;
  if (Hq < 0 || Hq % c->Hkv != 0) return SAGE_ERR_INVALID_ARG;
  std::memset(d, 0, sizeof(*d));
  if (Hq == 0 || b->B == 0) return SAGE_OK;
  d->group = Hq / c->Hkv;
  d->chunks = (d->group + 15) / 16;
  d->chunk_heads = (d->group + d->chunks - 1) / d->chunks;
  d->NT = d->chunk_heads > 8 ? 2 : 1;
  const int64_t pairs = static_cast<int64_t>(b->B) * c->Hkv * d->chunks;
  if (pairs >= (int64_t(1) << 26) || Hq > 65535) return SAGE_ERR_UNSUPPORTED;
  const int tile = sage::tile_keys(c->format == SAGE_CACHE_FP4, c->D);
  const int64_t tiles = std::max<int64_t>(1, (static_cast<int64_t>(b->table_width) * c->page_size + tile - 1) / tile);
  if (tiles * pairs >= (int64_t(1) << 38)) return SAGE_ERR_UNSUPPORTED;  // a share's tiles are counted in 32 bits
  d->max_grid = static_cast<int>(std::min<int64_t>(sage::kMaxDecodeCtas, pairs * (tiles + 1)));
  const size_t rows = static_cast<size_t>(d->max_grid) * 2 * 8 * d->NT;
  d->rec = up256(static_cast<size_t>(d->max_grid) * 16);
  d->ml = up256(rows * 8);
  d->o = up256(rows * c->D * 4);
  d->bytes = d->rec + d->ml + d->o;
  return SAGE_OK;
}

}  // namespace

extern "C" {

sage_status_t sage_fp4_norm_rope(const sage_fp4_rows_t* q, const sage_fp4_rows_t* k, int B, int N, int D,
                                 sage_dtype_t dtype, const sage_fp4_rope_t* rope, const int32_t* positions,
                                 void* stream) {
  if (B < 0 || N < 0 || !valid_dtype(dtype)) return SAGE_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return SAGE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * N >= (int64_t(1) << 31)) return SAGE_ERR_UNSUPPORTED;
  if (sage_status_t s = check_rope(rope, D); s != SAGE_OK) return s;
  if (B == 0 || N == 0) return SAGE_OK;
  for (const sage_fp4_rows_t* r : {q, k})
    if (sage_status_t s = check_rows(r, B, N, D); s != SAGE_OK) return s;
  if (positions != nullptr && !aligned(positions, 4)) return SAGE_ERR_INVALID_ARG;
  sage::RowsParams p;
  std::memset(&p, 0, sizeof(p));
  set_q(&p, q);
  if (k != nullptr && k->heads > 0) {
    p.Hk = k->heads;
    p.k = k->x;
    p.ko = k->y;
    p.sk = strides(k->x_stride);
    p.sko = strides(k->y_stride);
  }
  if (p.Hq == 0 && p.Hk == 0) return SAGE_OK;
  p.T = B * N;
  p.N = N;
  p.positions = positions;
  set_rope(&p, rope);
  if (int s = sage::device_error_word(&p.err); s != SAGE_OK) return static_cast<sage_status_t>(s);
  return static_cast<sage_status_t>(
      sage::status_of(sage::launch_rows(p, D, dtype, false, false, static_cast<cudaStream_t>(stream))));
}

sage_status_t sage_fp4_cache_append(const sage_fp4_cache_t* cache, const sage_fp4_batch_t* batch, const void* k,
                                    const int64_t k_stride[2], const void* v, const int64_t v_stride[2], int total,
                                    const sage_fp4_rope_t* rope, const sage_fp4_rows_t* q, void* stream) {
  if (sage_status_t s = check_cache(cache); s != SAGE_OK) return s;
  if (sage_status_t s = check_batch(cache, batch, true, total); s != SAGE_OK) return s;
  if (sage_status_t s = check_rope(rope, cache->D); s != SAGE_OK) return s;
  if (batch->B == 0 || total == 0) return SAGE_OK;
  if (sage_status_t s = check_rows(q, 1, total, cache->D); s != SAGE_OK) return s;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride == nullptr || v_stride == nullptr) return SAGE_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    if (!valid_stride(k_stride[i], 8) || !valid_stride(v_stride[i], 8)) return SAGE_ERR_INVALID_ARG;
  sage::RowsParams p;
  std::memset(&p, 0, sizeof(p));
  set_q(&p, q);
  p.Hk = p.Hv = cache->Hkv;
  p.k = k;
  p.v = v;
  p.sk = sage::Strides{0, k_stride[0], k_stride[1]};
  p.sv = sage::Strides{0, v_stride[0], v_stride[1]};
  p.T = p.N = total;
  set_rope(&p, rope);
  p.c = view_of(*cache, *batch);
  if (int s = sage::device_error_word(&p.err); s != SAGE_OK) return static_cast<sage_status_t>(s);
  return static_cast<sage_status_t>(sage::status_of(sage::launch_rows(
      p, cache->D, cache->dtype, true, cache->format == SAGE_CACHE_FP4, static_cast<cudaStream_t>(stream))));
}

sage_status_t sage_fp4_cache_gather(const sage_fp4_cache_t* cache, const sage_fp4_batch_t* batch, void* k,
                                    const int64_t k_stride[2], void* v, const int64_t v_stride[2], int total,
                                    void* stream) {
  if (sage_status_t s = check_cache(cache); s != SAGE_OK) return s;
  if (sage_status_t s = check_batch(cache, batch, true, total); s != SAGE_OK) return s;
  if (batch->B == 0 || total == 0) return SAGE_OK;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride == nullptr || v_stride == nullptr) return SAGE_ERR_INVALID_ARG;
  for (const int64_t* s : {k_stride, v_stride})
    if (!valid_stride(s[0], 8) || !valid_stride(s[1], 8) || !apart(s[0], cache->Hkv, cache->D) || !apart(s[1], total, cache->D))
      return SAGE_ERR_INVALID_ARG;
  sage::GatherParams p;
  std::memset(&p, 0, sizeof(p));
  p.k = k;
  p.v = v;
  p.sk = sage::Strides{0, k_stride[0], k_stride[1]};
  p.sv = sage::Strides{0, v_stride[0], v_stride[1]};
  p.T = total;
  p.c = view_of(*cache, *batch);
  if (int s = sage::device_error_word(&p.err); s != SAGE_OK) return static_cast<sage_status_t>(s);
  return static_cast<sage_status_t>(sage::status_of(sage::launch_gather(
      p, cache->D, cache->dtype, cache->format == SAGE_CACHE_FP4, static_cast<cudaStream_t>(stream))));
}

size_t sage_fp4_decode_workspace_bytes(const sage_fp4_cache_t* cache, const sage_fp4_batch_t* batch, int Hq) {
  DecodePlan d;
  return plan_decode(cache, batch, Hq, &d) == SAGE_OK ? d.bytes : 0;
}

sage_status_t sage_fp4_attn_decode(const sage_fp4_cache_t* cache, const sage_fp4_batch_t* batch, const void* q,
                                   const int64_t q_stride[2], void* out, const int64_t o_stride[2], int Hq,
                                   float sm_scale, void* workspace, size_t ws_bytes, void* stream) {
  DecodePlan d;
  if (sage_status_t s = plan_decode(cache, batch, Hq, &d); s != SAGE_OK) return s;
  if (!std::isfinite(sm_scale)) return SAGE_ERR_INVALID_ARG;
  if (d.max_grid == 0) return SAGE_OK;
  if (!aligned(q, 16) || !aligned(out, 16) || q_stride == nullptr || o_stride == nullptr) return SAGE_ERR_INVALID_ARG;
  const int64_t counts[2] = {batch->B, Hq};
  for (int i = 0; i < 2; ++i) {
    if (!valid_stride(q_stride[i], 8) || !valid_stride(o_stride[i], 8)) return SAGE_ERR_INVALID_ARG;
    if (!apart(o_stride[i], counts[i], cache->D)) return SAGE_ERR_INVALID_ARG;
    if (q == out && counts[i] > 1 && q_stride[i] != o_stride[i]) return SAGE_ERR_INVALID_ARG;
  }
  if (!aligned(workspace, 256) || ws_bytes < d.bytes) return SAGE_ERR_INVALID_ARG;
  sage::DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = q;
  p.out = out;
  p.sqb = q_stride[0];
  p.sqh = q_stride[1];
  p.sob = o_stride[0];
  p.soh = o_stride[1];
  p.Hq = Hq;
  p.group = d.group;
  p.chunks = d.chunks;
  p.chunk_heads = d.chunk_heads;
  const float scale = sm_scale > 0.0f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(cache->D));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.c = view_of(*cache, *batch);
  const int unit = cache->format == SAGE_CACHE_FP4 ? 32 : 8;  // elements in 16 bytes
  for (int i = 0; i < 3; ++i) {
    p.ku[i] = static_cast<uint32_t>(cache->k_stride[i] / unit);
    p.vu[i] = static_cast<uint32_t>(cache->v_stride[i] / unit);
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.rec = reinterpret_cast<int4*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + d.rec);
  p.part_o = reinterpret_cast<float*>(ws + d.rec + d.ml);
  if (int s = sage::device_error_word(&p.err); s != SAGE_OK) return static_cast<sage_status_t>(s);
  return static_cast<sage_status_t>(sage::status_of(sage::launch_decode(
      p, cache->D, cache->dtype, cache->format == SAGE_CACHE_FP4, d.NT, d.max_grid, static_cast<cudaStream_t>(stream))));
}

}  // extern "C"
