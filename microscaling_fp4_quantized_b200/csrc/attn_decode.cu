// Attention of one query token per sequence over a paged cache (sm_100a).
//
//   out[b, h] = sum_n p_n v_n / sum_n p_n,  p_n = exp(sm_scale q[b, h] . k_n - m),  n < seq_lens[b]
//
// Bound: every cached key and value is read once for all query heads that share it, 4 D bytes a
// token and head (FP4: 1.125 D), against 4 D flops per query head: with up to 16 query heads per
// key/value head the tensor rate needed at the full memory rate is under a twentieth of the
// chip's, so HBM is the floor.
//
// Work split. The tokens of all (sequence, key/value head) pairs are cut into 64-key tiles, laid
// end to end and dealt to the CTAs in equal contiguous shares, so that neither ragged lengths nor
// few pairs leave SMs idle. A CTA finishes the pairs that lie inside its share and leaves
// the (at most two) that cross its borders as partial (max, sum, output) triples;
// join_kernel adds those up in the order of the shares, so results do not depend on timing.
//
// Each of the four warps owns 16 keys of a tile and its own ring of cp.async stages, so
// the main loop has no block barrier; the warps meet when a pair ends. Scores are formed
// transposed, S^T = K Q^T with 16 keys by 8 query heads per mma.m16n8k16 (a tcgen05 tile has 128 rows,
// of which a decode step fills at most 16): a group of 8 heads wastes nothing, and movmatrix turns S^T
// into the operand of O^T = V^T P^T. The running maximum is raised only when a score exceeds it by
// 2^4, checked by one vote per tile: probabilities then reach 2^4 times the scale they are kept at.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "paged.h"
#include "sm100_ptx.cuh"

namespace sage {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpKeys = kTileKeys / kWarps;  // 16
// Probabilities are kept as 2^kShift exp2(s - m): fp16 then keeps 11 bits for weights down to 2^-22
// of the maximum, and the largest (2^kShift 2^4) is far from its limit. The factor cancels in the end.
constexpr float kShift = 8.0f, kSlack = 4.0f;

template <typename T>
struct Is {
  static constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(valid ? N : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}

// Two E4M3 bytes -> two fp16 values.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Probabilities of two heads as one operand word, and the values that the rounding left: the
// denominator sums those, so that the weights of the sum that is formed add up to one.
template <bool BF16>
__device__ __forceinline__ uint32_t pack_p(float& a, float& b) {
  uint32_t r;
  if constexpr (BF16) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    a = __uint_as_float(r << 16);
    b = __uint_as_float(r & 0xFFFF0000u);
  } else {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
    a = f.x;
    b = f.y;
  }
  return r;
}

// Shared memory of a CTA: per warp kStages stages of 16 keys' K and V (FP4: codes of K, codes of
// V, scales of K, scales of V), then the meeting area of the warps.
template <int D, bool FP4>
struct Smem {
  static constexpr int kKey = FP4 ? D / 2 : 2 * D;  // bytes of a key's codes or elements
  static constexpr int kSf = FP4 ? D / 16 : 0;
  static constexpr int kV = kWarpKeys * kKey;                             // offsets in a stage
  [[maybe_unused]] static constexpr int kKs = 2 * kV, kVs = kKs + kWarpKeys * kSf;
  static constexpr int kStage = 2 * kWarpKeys * (kKey + kSf);
  static constexpr int kStages = FP4 ? 4 : (D == 128 ? 3 : 4);
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kRow = D + 4;  // floats of a head's row in the meeting area
  static constexpr int kMeet = kWarps * 8 * kRow * 4;
  static constexpr int kBytes = kRing + kMeet + kWarps * 8 * 2 * 4;  // 112.8 KB at most: two CTAs per SM
};

// Row of the V codes' stage that key `key` takes: a lane's keys 2t, 2t+1, 2t+8, 2t+9 lie in rows
// t, 4+t, 8+t, 12+t, so the four lanes of a quad read consecutive rows (with the chunk
// swizzle of D = 128, every read is free of bank conflicts).
__device__ __forceinline__ int v_row(int key) { return (key & 8) | ((key & 1) << 2) | ((key >> 1) & 3); }

// FP4 path: the query row's share of this lane (D / 4 channels from t4 * D / 4 on, two operand words per
// step of four) in fp16. The row is scaled by a power of two that brings its maximum into [2^14, 2^15),
// which is exact but for elements more than 2^28 below it; undo[] = the inverse factors of the
// two heads whose scores this lane holds.
template <typename T, int KS>
__device__ __forceinline__ void load_q_fp16(const T* q, bool valid, int t4, uint32_t (&qf)[KS][2], float (&undo)[2]) {
  float x[KS * 4];
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < KS / 2; ++i) {
    const uint4 raw = valid ? __ldg(reinterpret_cast<const uint4*>(q + t4 * (KS * 4)) + i) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (Is<T>::bf16) {
        x[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
        x[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
        x[8 * i + 2 * e] = f.x;
        x[8 * i + 2 * e + 1] = f.y;
      }
      mx = fmaxf(mx, fmaxf(fabsf(x[8 * i + 2 * e]), fabsf(x[8 * i + 2 * e + 1])));
    }
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const uint32_t ex = max(__float_as_uint(mx) >> 23, 16u);  // biased exponent; tiny rows stop at 2^127
  const float f = __uint_as_float((268u - ex) << 23), inv = __uint_as_float((ex - 14u) << 23);
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    qf[k][0] = pack_half2(x[4 * k] * f, x[4 * k + 1] * f);
    qf[k][1] = pack_half2(x[4 * k + 2] * f, x[4 * k + 3] * f);
  }
  undo[0] = __shfl_sync(0xffffffffu, inv, 8 * t4);
  undo[1] = __shfl_sync(0xffffffffu, inv, 8 * t4 + 4);
}

// S^T of 16 FP4 keys. The order of a contraction is free as long as both operands share it: lane
// (r, t4) takes channels t4 D/4 .. of keys r and r + 8, one or two whole scale blocks, and
// step k contracts channels 4k .. 4k+3 of each lane's range.
template <int D, int NT>
__device__ __forceinline__ void scores_fp4(uint32_t stage, int r, int t4, const uint32_t (&qf)[NT][D / 16][2], float (&s)[NT][4]) {
  using S = Smem<D, true>;
  constexpr int W = D / 32;  // code words of a lane and key: 4 or 2
  uint32_t w[2][W], sc[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int key = r + 8 * half;
    const uint32_t sf = stage + S::kKs + key * S::kSf;
    if constexpr (D == 128) {
      const uint4 v = lds128(stage + key * S::kKey + t4 * 16);
      w[half][0] = v.x; w[half][1] = v.y; w[half][2] = v.z; w[half][3] = v.w;
      sc[half] = e4m3x2_to_f16x2(lds16(sf + 2 * t4));
    } else {
      const uint2 v = lds64(stage + key * S::kKey + t4 * 8);
      w[half][0] = v.x; w[half][1] = v.y;
      sc[half] = e4m3x2_to_f16x2(lds8(sf + t4));
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    uint32_t v0[4], v1[4];
    e2m1x8_to_f16x2(w[0][i], v0);
    e2m1x8_to_f16x2(w[1][i], v1);
    const uint32_t sel = i < 2 ? 0x1010u : 0x3232u;  // the block of the word's 8 channels
    const uint32_t s0 = __byte_perm(sc[0], 0, sel), s1 = __byte_perm(sc[1], 0, sel);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a[4] = {mul_f16x2(v0[2 * h], s0), mul_f16x2(v1[2 * h], s1), mul_f16x2(v0[2 * h + 1], s0),
                             mul_f16x2(v1[2 * h + 1], s1)};
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16816<false>(s[n], a, qf[n][2 * i + h][0], qf[n][2 * i + h][1]);
    }
  }
}

// O^T += V^T P^T over 16 FP4 keys. Lane (r, t4) takes channels r D/8 .. of keys 2t, 2t+1, 2t+8, 2t+9;
// the operand wants two keys' values of one channel side by side, so the nibbles of two
// keys are interleaved before they are decoded.
template <int D, int NT>
__device__ __forceinline__ void values_fp4(uint32_t stage, int r, int t4, const uint32_t (&pb)[NT][2], float (&o)[NT][D / 16][4]) {
  using S = Smem<D, true>;
  constexpr int W = D / 64;  // code words of a lane and key: 2 or 1
  uint32_t w[4][W], sc[2];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t row = stage + S::kV + (4 * e + t4) * S::kKey;
    if constexpr (D == 128) {
      const uint2 v = lds64(row + (((r >> 1) ^ (t4 & 2)) << 4) + (r & 1) * 8);
      w[e][0] = v.x; w[e][1] = v.y;
    } else {
      w[e][0] = lds32(row + r * 4);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t sf = stage + S::kVs + (8 * h + 2 * t4) * S::kSf + (D == 128 ? r : r >> 1);
    sc[h] = e4m3x2_to_f16x2(lds8(sf) | lds8(sf + S::kSf) << 8);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    uint32_t lo[2][4], hi[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a = w[2 * h][i], b = w[2 * h + 1][i];
      e2m1x8_to_f16x2((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), lo[h]);
      e2m1x8_to_f16x2(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), hi[h]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a[4] = {mul_f16x2(lo[0][e], sc[0]), mul_f16x2(hi[0][e], sc[0]), mul_f16x2(lo[1][e], sc[1]),
                             mul_f16x2(hi[1][e], sc[1])};
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16816<false>(o[n][4 * i + e], a, pb[n][0], pb[n][1]);
    }
  }
}

// acc / sum (no keys: 0), rounded once.
template <typename T, int N>
__device__ __forceinline__ void store_out(T* out, const float (&acc)[N], float sum) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint32_t w[N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    if constexpr (Is<T>::bf16) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      w[e] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      w[e] = pack_half2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    }
  }
  if constexpr (N == 8) *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
}

// Tiles of a sequence: at least one, so that empty sequences too get their (zero) output.
__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + kTileKeys - 1) / kTileKeys : 1; }

__device__ __forceinline__ int length_of(const CacheView& c, int b, uint32_t* err) {
  const int len = __ldg(c.lens + b);
  if (len >= 0 && len <= c.capacity) return len;
  if (err != nullptr) atomicOr(err, kDevErrSeqlens);
  return len < 0 ? 0 : c.capacity;
}

// Tiles of all sequences (of one head chunk), and in `mine` those before this thread's range of
// ceil(B / kThreads) sequences; by the whole block.
__device__ __forceinline__ int64_t count_tiles(const CacheView& c, int64_t* red, int64_t* mine, uint32_t* err) {
  const int per = (c.B + kThreads - 1) / kThreads, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int lo = min(c.B, static_cast<int>(threadIdx.x) * per), hi = min(c.B, lo + per);
  int64_t s = 0;
  for (int b = lo; b < hi; ++b) s += tiles_of(length_of(c, b, err));
  int64_t inc = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) red[w] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) before += red[i];
    all += red[i];
  }
  *mine = before + inc - s;
  return all;
}

// First tile of CTA i's share of W tiles.
__device__ __forceinline__ int64_t share(int64_t W, int i, int grid) { return W * i / grid; }

// Place in the row of tiles: sequence, head chunk, tile.
struct Cursor {
  int b, hc, t, len, nt;
};

}  // namespace

template <typename T, int D, int NT, bool FP4>
__global__ void __launch_bounds__(kThreads, FP4 && NT == 1 ? 4 : 2) decode_kernel(const DecodeParams p) {
  using S = Smem<D, FP4>;
  constexpr bool kMmaBf16 = Is<T>::bf16 && !FP4;  // FP4 values are exact in fp16
  constexpr int KS = D / 16;                      // contraction steps of S^T, channel tiles of O^T
  extern __shared__ __align__(16) uint8_t smem[];
  float* meet = reinterpret_cast<float*>(smem + S::kRing);
  float* meet_ml = meet + kWarps * 8 * S::kRow;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, t4 = lane & 3;
  const CacheView& c = p.c;
  const int HC = c.Hkv * p.chunks;

  // This CTA's share, and where it begins.
  int64_t before;
  __shared__ int64_t s_red[kWarps];
  __shared__ int s_b;
  __shared__ int64_t s_before;
  const int64_t W = count_tiles(c, s_red, &before, blockIdx.x == 0 ? p.err : nullptr) * HC;
  const int64_t u0 = share(W, blockIdx.x, p.grid), u1 = share(W, blockIdx.x + 1, p.grid);
  if (u0 >= u1) {  // uniform over the block. Fewer tiles than CTAs: a join skips the empty shares
    if (tid < 8 * NT) {
      float* ml = p.part_ml + (static_cast<int64_t>(blockIdx.x) * 2 * (8 * NT) + tid) * 2;
      ml[0] = -INFINITY;
      ml[1] = 0.0f;
    }
    return;
  }
  {
    const int per = (c.B + kThreads - 1) / kThreads;
    const int lo = min(c.B, tid * per), hi = min(c.B, lo + per);
    for (int b = lo; b < hi; ++b) {
      const int64_t n = tiles_of(length_of(c, b, nullptr));
      if (before * HC <= u0 && u0 < (before + n) * HC) {
        s_b = b;
        s_before = before;
      }
      before += n;
    }
  }
  __syncthreads();
  Cursor pc;  // where the copies are
  pc.b = s_b;
  pc.len = length_of(c, pc.b, nullptr);
  pc.nt = tiles_of(pc.len);
  {
    const int64_t in = u0 - s_before * HC;
    pc.hc = static_cast<int>(in / pc.nt);
    pc.t = static_cast<int>(in - static_cast<int64_t>(pc.hc) * pc.nt);
  }
  Cursor cc = pc;  // where the arithmetic is
  const int count = static_cast<int>(u1 - u0);

  auto advance = [&](Cursor& x) {
    if (++x.t < x.nt) return;
    x.t = 0;
    if (++x.hc < HC) return;
    x.hc = 0;
    if (++x.b < c.B) {
      x.len = length_of(c, x.b, nullptr);
      x.nt = tiles_of(x.len);
    }
  };
  // The page of this lane's key (lanes 0-15: for K, 16-31: the same keys, for V), loaded one tile ahead.
  auto page_of = [&](const Cursor& x) -> int {
    const int pos = x.t * kTileKeys + warp * kWarpKeys + (lane & 15);
    if (pos >= x.len) return -1;
    const int page = __ldg(c.table + x.b * c.table_stride + div_by_page(c.page, pos));
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(c.num_pages)) {
      atomicOr(p.err, kDevErrPages);
      return -1;
    }
    return page;
  };
  const uint32_t ring = smem_u32(smem) + warp * (S::kStages * S::kStage);
  const Strides st = lane < 16 ? c.sk : c.sv;
  auto copy_tile = [&](const Cursor& x, int page, uint32_t stage) {
    const int k0 = x.t * kTileKeys + warp * kWarpKeys;
    if (k0 >= x.len) return;
    // Lane l's key as a row offset in units of 16 bytes; bit-all-ones: no such key.
    const uint32_t pos = k0 + (lane & 15);
    const uint32_t slot = pos - div_by_page(c.page, pos) * c.page.d;
    uint32_t off = 0xffffffffu;
    if (page >= 0) {
      const int64_t el = page * st.b + static_cast<int64_t>(x.hc / p.chunks) * st.h + static_cast<int64_t>(slot) * st.n;
      off = static_cast<uint32_t>(el / (FP4 ? 32 : 8));
    }
    constexpr int CPK = S::kKey / 16, KPI = 32 / CPK;  // 16-byte chunks per key, keys per instruction
    const int ch = lane % CPK;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const char* base = static_cast<const char*>(half ? c.v : c.k);
      const uint32_t dst = stage + half * S::kV;
#pragma unroll
      for (int i = 0; i < kWarpKeys / KPI; ++i) {
        const int key = i * KPI + lane / CPK;
        const uint32_t o = __shfl_sync(0xffffffffu, off, half * 16 + key);
        const bool valid = o != 0xffffffffu;
        uint32_t at;
        if constexpr (!FP4) {
          at = key * S::kKey + ((ch ^ (key & 7)) << 4);
        } else if (half == 0) {
          at = key * S::kKey + (ch << 4);
        } else {
          const int row = v_row(key);
          at = row * S::kKey + ((D == 128 ? ch ^ (row & 2) : ch) << 4);
        }
        cp_async16(dst + at, base + (valid ? static_cast<uint64_t>(o) * 16 : 0) + ch * 16, valid);
      }
    }
    if constexpr (FP4) {
      const bool valid = off != 0xffffffffu;
      const uint8_t* sf = lane < 16 ? c.k_sf : c.v_sf;
      cp_async_small<S::kSf>(stage + S::kKs + lane * S::kSf, sf + (valid ? static_cast<uint64_t>(off) * 2 : 0), valid);
    }
  };

  int page = page_of(pc);
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) {
    if (i < count) {
      copy_tile(pc, page, ring + i * S::kStage);
      advance(pc);
      if (i + 1 < count) page = page_of(pc);
    }
    cp_async_commit();
  }

  uint32_t qf[NT][KS][2];
  float o[NT][KS][4], m[NT][2], l[NT][2], qs[NT][2];
  uint32_t slot = 0, fill = S::kStages - 1;  // stages to read and to refill
  bool first = true;
  for (int i = 0; i < count; ++i) {
    const int hk = cc.hc / p.chunks, chunk = cc.hc - hk * p.chunks;
    const int head0 = hk * p.group + chunk * p.chunk_heads;
    const int heads = min(p.chunk_heads, p.group - chunk * p.chunk_heads);
    if (first) {  // a new pair: its queries
      first = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int h = n * 8 + r;
        const T* q = static_cast<const T*>(p.q) + cc.b * p.sqb + static_cast<int64_t>(head0 + (h < heads ? h : 0)) * p.sqh;
        float sc[2] = {1.0f, 1.0f};
        if constexpr (!FP4) {
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * t4);
            qf[n][s][0] = h < heads ? __ldg(w) : 0u;
            qf[n][s][1] = h < heads ? __ldg(w + 4) : 0u;
          }
        } else {
          load_q_fp16<T, KS>(q, h < heads, t4, qf[n], sc);
        }
        qs[n][0] = p.scale_log2 * sc[0];
        qs[n][1] = p.scale_log2 * sc[1];
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][s][e] = 0.0f;
      }
    }
    cp_async_wait<S::kStages - 2>();
    __syncwarp();  // this tile has arrived for every lane, and every lane has read the one before
    if (i + S::kStages - 1 < count) {
      copy_tile(pc, page, ring + fill * S::kStage);
      advance(pc);
      if (i + S::kStages < count) page = page_of(pc);
    }
    cp_async_commit();
    const int k0 = cc.t * kTileKeys + warp * kWarpKeys;
    if (k0 < cc.len) {
      const uint32_t stage = ring + slot * S::kStage;
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
      if constexpr (!FP4) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int key = (lane & 7) + (lane & 8), ch = 2 * k + (lane >> 4);
          uint32_t a[4];
          ldsm4(stage + key * S::kKey + ((ch ^ (key & 7)) << 4), a);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<kMmaBf16>(s[n], a, qf[n][k][0], qf[n][k][1]);
        }
      } else {
        scores_fp4<D, NT>(stage, r, t4, qf, s);
      }
      const bool ok0 = k0 + r < cc.len, ok1 = k0 + 8 + r < cc.len;
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = (e < 2 ? ok0 : ok1) ? s[n][e] * qs[n][e & 1] : -INFINITY;
        raise |= fmaxf(s[n][0], s[n][2]) > m[n][0] + kSlack || fmaxf(s[n][1], s[n][3]) > m[n][1] + kSlack;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[n][e], s[n][e + 2]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x = fmaxf(x, m[n][e]);
            const float f = m[n][e] == -INFINITY ? 0.0f : ex2_approx(m[n][e] - x);
            m[n][e] = x;
            l[n][e] *= f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[n][k][e] *= f;
              o[n][k][e + 2] *= f;
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[n][e & 1] == -INFINITY ? 0.0f : m[n][e & 1];
          s[n][e] = ex2_approx(s[n][e] - ref + kShift);
        }
        pb[n][0] = pack_p<kMmaBf16>(s[n][0], s[n][1]);
        pb[n][1] = pack_p<kMmaBf16>(s[n][2], s[n][3]);
        l[n][0] += s[n][0] + s[n][2];
        l[n][1] += s[n][1] + s[n][3];
        pb[n][0] = movm_t(pb[n][0]);
        pb[n][1] = movm_t(pb[n][1]);
      }
      if constexpr (!FP4) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int key = (lane & 7) + ((lane & 16) >> 1), ch = 2 * k + ((lane >> 3) & 1);
          uint32_t a[4];
          ldsm4_t(stage + S::kV + key * S::kKey + ((ch ^ (key & 7)) << 4), a);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<kMmaBf16>(o[n][k], a, pb[n][0], pb[n][1]);
        }
      } else {
        values_fp4<D, NT>(stage, r, t4, pb, o);
      }
    }
    slot = slot + 1 == S::kStages ? 0 : slot + 1;
    fill = fill + 1 == S::kStages ? 0 : fill + 1;

    const Cursor at = cc;
    advance(cc);
    if (at.t + 1 < at.nt && i + 1 < count) continue;
    // The pair ends, here or with this share: the warps meet.
    first = true;
    const bool whole = at.t + 1 == at.nt && at.t <= i;  // its first tile was tile i - at.t of this share
    // Partial 0: a pair that began before this share; partial 1: one that only goes on after it.
    const int part = at.t > i ? 0 : 1;
    if (tid == 0) {
      // What join_kernel has to do, one record per pair (by the CTA with the pair's first tile) or, when
      // there are more pairs than CTAs, one per CTA (for the pair that goes on after it).
      const bool by_pair = p.joins < p.grid;
      if (by_pair ? part == 1 : i + 1 == count) {
        int4 rec = make_int4(-1, 0, 0, 0);
        if (part == 1 && !whole) {
          const int64_t end = u0 + i - at.t + at.nt;  // past the pair's last tile
          rec = make_int4(at.b, at.hc, static_cast<int>(blockIdx.x), static_cast<int>((end * p.grid - 1) / W));
        }
        p.rec[by_pair ? static_cast<int64_t>(at.b) * HC + at.hc : blockIdx.x] = rec;
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
      }
      __syncthreads();  // the area's last readers are done
      if (r == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          meet_ml[(warp * 8 + 2 * t4 + e) * 2] = m[n][e];
          meet_ml[(warp * 8 + 2 * t4 + e) * 2 + 1] = l[n][e];
        }
      }
      float* row = meet + (warp * 8 + 2 * t4) * S::kRow;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        // Channels of a tile's two rows: neighbours of the lane's own range in FP4, else 8 apart.
        const int ch = FP4 ? (D / 8) * r + 2 * k : 16 * k + r;
        constexpr int step = FP4 ? 1 : 8;
        row[ch] = o[n][k][0];
        row[S::kRow + ch] = o[n][k][1];
        row[ch + step] = o[n][k][2];
        row[S::kRow + ch + step] = o[n][k][3];
      }
      __syncthreads();
      // 16 threads per head, D / 16 channels each.
      const int h = tid >> 4, c0 = (tid & 15) * (D / 16);
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, meet_ml[(w * 8 + h) * 2]);
      float acc[D / 16], sum = 0.0f;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) acc[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = meet_ml[(w * 8 + h) * 2];
        const float f = mw == -INFINITY ? 0.0f : ex2_approx(mw - mx);
        sum += meet_ml[(w * 8 + h) * 2 + 1] * f;
        const float* src = meet + (w * 8 + h) * S::kRow + c0;
#pragma unroll
        for (int e = 0; e < D / 16; e += 4) {
          const float4 v = *reinterpret_cast<const float4*>(src + e);
          acc[e] += v.x * f;
          acc[e + 1] += v.y * f;
          acc[e + 2] += v.z * f;
          acc[e + 3] += v.w * f;
        }
      }
      if (n * 8 + h < heads) {
        if (whole) {
          T* out = static_cast<T*>(p.out) + at.b * p.sob + static_cast<int64_t>(head0 + n * 8 + h) * p.soh + c0;
          store_out<T, D / 16>(out, acc, sum);
        } else {
          const int64_t g = (static_cast<int64_t>(blockIdx.x) * 2 + part) * (8 * NT) + n * 8 + h;
          float* po = p.part_o + g * D + c0;
#pragma unroll
          for (int e = 0; e < D / 16; e += 4) *reinterpret_cast<float4*>(po + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
          if ((tid & 15) == 0) {
            p.part_ml[g * 2] = mx;
            p.part_ml[g * 2 + 1] = sum;
          }
        }
      }
    }
  }
}

// Adds up the partial results of the pairs that lie in more than one share. Block (record, head);
// 8 groups of 16 threads take every eighth share each, then meet.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(128) join_kernel(const DecodeParams p) {
  constexpr int N = D / 16;
  __shared__ float s_acc[8][D];
  __shared__ float s_ml[8][2];
  const int tid = threadIdx.x, g = tid >> 4, c0 = (tid & 15) * N, h = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 rec = p.rec[blockIdx.x];
  if (rec.x < 0) return;
  const int hk = rec.y / p.chunks, chunk = rec.y - hk * p.chunks;
  if (h >= min(p.chunk_heads, p.group - chunk * p.chunk_heads)) return;
  auto row_of = [&](int cta) { return (static_cast<int64_t>(cta) * 2 + (cta == rec.z ? 1 : 0)) * (8 * NT) + h; };
  // The group's maximum first: the sums then need no rescaling.
  float mx = -INFINITY;
  for (int cta = rec.z + g; cta <= rec.w; cta += 8) mx = fmaxf(mx, p.part_ml[row_of(cta) * 2]);
  float acc[N], sum = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.0f;
#pragma unroll 4
  for (int cta = rec.z + g; cta <= rec.w; cta += 8) {
    const int64_t row = row_of(cta);
    const float m = p.part_ml[row * 2];
    if (m == -INFINITY) continue;  // an empty share has no output
    const float f = ex2_approx(m - mx);
    sum += p.part_ml[row * 2 + 1] * f;
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + row * D + c0 + e);
      acc[e] += v.x * f;
      acc[e + 1] += v.y * f;
      acc[e + 2] += v.z * f;
      acc[e + 3] += v.w * f;
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) s_acc[g][c0 + e] = acc[e];
  if ((tid & 15) == 0) {
    s_ml[g][0] = mx;
    s_ml[g][1] = sum;
  }
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = fmaxf(mx, s_ml[i][0]);
  sum = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float m = s_ml[i][0];
    const float f = m == -INFINITY ? 0.0f : ex2_approx(m - mx);
    sum += s_ml[i][1] * f;
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] += s_acc[i][c0 + e] * f;
  }
  const int64_t head = static_cast<int64_t>(hk) * p.group + chunk * p.chunk_heads + h;
  store_out<T, N>(static_cast<T*>(p.out) + rec.x * p.sob + head * p.soh + c0, acc, sum);
}

namespace {

constexpr int kMaxDevices = 64;

// CTAs of the kernel that fit the device, asked once per device (and the kernel's shared
// memory limit raised then); 0 on an error.
template <auto kernel>
int resident_ctas(int smem, cudaError_t* e) {
  static std::mutex mu;
  static int known[kMaxDevices] = {};
  int dev = 0;
  if ((*e = cudaGetDevice(&dev)) != cudaSuccess) return 0;
  if (dev < 0 || dev >= kMaxDevices) {
    *e = cudaErrorInvalidDevice;
    return 0;
  }
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev] == 0) {
    int sms = 0, per = 0;
    if ((*e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return 0;
    if ((*e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return 0;
    if ((*e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, smem)) != cudaSuccess) return 0;
    if (per < 1) {
      *e = cudaErrorLaunchOutOfResources;
      return 0;
    }
    known[dev] = sms * per;
  }
  return known[dev];
}

template <typename T, int D, int NT, bool FP4>
cudaError_t launch_one(DecodeParams p, int max_grid, cudaStream_t stream) {
  constexpr int smem = Smem<D, FP4>::kBytes;
  cudaError_t e = cudaSuccess;
  const int fit = resident_ctas<decode_kernel<T, D, NT, FP4>>(smem, &e);
  if (e != cudaSuccess) return e;
  p.grid = max_grid < fit ? max_grid : fit;
  const int64_t pairs = static_cast<int64_t>(p.c.B) * p.c.Hkv * p.chunks;
  p.joins = static_cast<int>(pairs < p.grid ? pairs : p.grid);
  decode_kernel<T, D, NT, FP4><<<p.grid, kThreads, smem, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.c.capacity <= kTileKeys) return cudaSuccess;  // one tile per pair: none is split
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.joins, p.chunk_heads);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, D, NT>, p);
}

template <typename T>
cudaError_t launch_type(const DecodeParams& p, int D, bool fp4, int NT, int max_grid, cudaStream_t stream) {
  if (D == 128) {
    if (fp4) return NT == 1 ? launch_one<T, 128, 1, true>(p, max_grid, stream) : launch_one<T, 128, 2, true>(p, max_grid, stream);
    return NT == 1 ? launch_one<T, 128, 1, false>(p, max_grid, stream) : launch_one<T, 128, 2, false>(p, max_grid, stream);
  }
  if (fp4) return NT == 1 ? launch_one<T, 64, 1, true>(p, max_grid, stream) : launch_one<T, 64, 2, true>(p, max_grid, stream);
  return NT == 1 ? launch_one<T, 64, 1, false>(p, max_grid, stream) : launch_one<T, 64, 2, false>(p, max_grid, stream);
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& p, int D, int dtype, bool fp4, int NT, int max_grid, cudaStream_t stream) {
  return dtype == kDtypeBF16 ? launch_type<__nv_bfloat16>(p, D, fp4, NT, max_grid, stream)
                             : launch_type<__half>(p, D, fp4, NT, max_grid, stream);
}

}  // namespace sage
