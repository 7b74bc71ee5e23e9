// Launch interfaces of the paged cache kernels (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "sage_internal.h"

namespace sage {

// n / d for 0 <= n < 2^31 by a multiply: with L = ceil(log2 d) and m = floor(2^(31+L) / d) + 1,
// m d lies in (2^(31+L), 2^(31+L) + d], d <= 2^L, so n m / 2^(31+L) exceeds n / d by less than
// n 2^L / (d 2^(31+L)) < 1 / d and has the same integer part.
struct FastDiv {
  uint32_t d, m, s;
};

inline FastDiv fast_div(uint32_t d) {
  uint32_t L = 0;
  while ((uint64_t(1) << L) < d) ++L;
  const unsigned __int128 m = ((unsigned __int128)1 << (31 + L)) / d + 1;
  return FastDiv{d, static_cast<uint32_t>(m), 31 + L};
}

__device__ __forceinline__ uint32_t div_by_page(const FastDiv& f, uint32_t n) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * f.m) >> f.s);
}

struct CacheView {
  void *k, *v;
  uint8_t *k_sf, *v_sf;
  Strides sk, sv;  // elements of (page, head, slot)
  int num_pages, Hkv;
  FastDiv page;
  const int32_t* table;
  int64_t table_stride;
  int capacity;  // table_width * page_size
  const int32_t* lens;
  const int32_t* cu;
  int B;
};

// Norm, rotation, append: token rows of up to three sets of heads.
struct RowsParams {
  const void *q, *k, *v;
  void *qo, *ko;         // dense outputs (ko unused when keys go to the cache)
  Strides sq, sk, sv, sqo, sko;
  int Hq, Hk, Hv;        // heads of each set (0: none)
  int T, N;              // tokens in all; tokens per sequence (dense), T for packed ones
  int items_q, items_k, items_v;  // items along the heads of each set (set by launch_rows)
  int per_q, per_k, per_v;        // heads of an item
  const void *qw, *kw;
  int w32;
  float eps;
  const float* rope;
  int rope_len, R, interleaved;
  const int32_t* positions;
  float minus_zero;               // -0, unknown to the compiler (set by launch_rows; see rows_kernel)
  CacheView c;
  uint32_t* err;
};

struct GatherParams {
  void *k, *v;
  Strides sk, sv;  // (unused, head, token)
  int T, heads_per_item, items;
  CacheView c;
  uint32_t* err;
};

struct DecodeParams {
  const void* q;
  void* out;
  int64_t sqb, sqh, sob, soh;
  int Hq, group;       // query heads per key/value head
  int chunks;          // chunks of the group, each with at most 8 * NT heads
  int chunk_heads;     // query heads of a chunk (the last one may have fewer)
  float scale_log2;    // sm_scale * log2(e)
  CacheView c;
  uint32_t ku[3], vu[3];  // strides of (page, head, slot) in units of 16 bytes of codes or elements
  float* part_o;       // [grid, 2, 8 * NT, D]
  float* part_ml;      // [grid, 2, 8 * NT, 2]
  int4* rec;           // [joins] what is to be joined
  int run;             // a warp's keys are consecutive in memory (set by launch_decode)
  int grid, joins, cluster, side;  // (set by launch_decode; side: blocks that share a range of tokens, one per head)
  uint32_t* err;
};

// Launches of these kernels may begin while the stream's last kernel drains (programmatic dependent
// launch; about 2 us less per call in a stream of them). Each waits for it first, before anything is read or
// written.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename P>
inline cudaError_t launch_dependent(void (*kernel)(P), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                                    const P& p, unsigned cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Keys of a CTA tile of the decode kernel: four warps with 16 (16-bit, D = 128), 32, or 64 each (FP4, D = 64,
// whose bytes per key are the fewest for the same work around them).
__host__ __device__ constexpr int tile_keys(bool fp4, int D) { return fp4 ? (D == 64 ? 256 : 128) : D == 64 ? 128 : 64; }
constexpr int kMaxDecodeCtas = 1184;  // 8 per SM: bound of the decode grid and of its workspace

cudaError_t launch_rows(const RowsParams& p, int D, int dtype, bool to_cache, bool fp4, cudaStream_t stream);
cudaError_t launch_gather(const GatherParams& p, int D, int dtype, bool fp4, cudaStream_t stream);
// NT: 8-head column tiles per chunk (1 or 2). max_grid bounds the grid and the partials.
cudaError_t launch_decode(const DecodeParams& p, int D, int dtype, bool fp4, int NT, int max_grid, cudaStream_t stream);

}  // namespace sage
