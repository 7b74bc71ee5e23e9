// Attention of one query token per sequence over a paged cache (sm_100a).
//
//   out[b, h] = sum_n p_n v_n / sum_n p_n,  p_n = exp(sm_scale q[b, h] . k_n - m),  n < seq_lens[b]
//
// Bound: every cached key and value is read once for all query heads that share it, 4 D bytes a
// token and head (FP4: 1.125 D), against 4 D flops per query head. 16-bit caches: with up to 16 query
// heads per key/value head the tensor rate needed at the full memory rate is under a twentieth of the
// chip's, so HBM is the bound. FP4 caches have the same floor, but need up to 57 flops a byte and, before
// them, every code in fp16: their bound is the instructions below.
//
// Work split. The tokens of all (sequence, key/value head) pairs are cut into tiles, laid end to
// end and dealt to the CTAs (as many as fit the machine) in contiguous shares of equal cost, so
// that neither ragged lengths nor few pairs leave SMs idle. Where the heads fill the machine evenly
// the shares are of one head's tiles instead, and the CTAs of all heads with the same share run side
// by side (see launch_one). A CTA finishes the pairs that lie inside its share and leaves the (at
// most two) that cross its borders as parts (maximum, sum of weights, average); join_kernel weighs
// those in the order of the shares, so results do not depend on timing. Small problems (see
// launch_one) take a cluster of up to 8 CTAs per pair instead, which joins its parts through
// distributed shared memory, in one launch.
//
// Each of the four warps owns 16, 32 or 64 keys of a tile and its own ring of cp.async stages, so
// the main loop has no block barrier; the warps meet when a pair ends. Scores are formed transposed,
// S^T = K Q^T with 16 keys by 8 query heads per mma.m16n8k16 (a tcgen05 tile has 128 rows, of which a
// decode step fills at most 16): a group of 8 heads wastes nothing, and movmatrix turns S^T into
// the operand of O^T = V^T P^T. The running maximum is raised only when a score exceeds it by
// 2^4, checked by one vote per tile: probabilities then reach 2^4 times the scale they are kept at.
//
// Measured on several B200s, joins included, share of the 6549 GB/s a copy reaches: 16-bit, 16 sequences of
// 256 to 16384 tokens, 32 heads on 8, D 128: 81 to 84 us, 6.0 to 6.2 TB/s (0.92 to 0.95), 128 heads on 8 88 us.
// 16-bit, 8 sequences of 2000 to 8192, 16 heads, D 64: 32.2 us, 5.2 TB/s (0.80). FP4, 64 sequences of 128 to
// 8192, heads on 8: D 128 32 heads 80 to 86 us (0.58 to 0.62), 64 heads 90 (0.56), 128 heads 131 (0.38), D 64
// 32 heads 52 us (0.48); one sequence of 131071, D 128: 41 to 42 us, 3.6 TB/s (0.56). FP4 waits for the
// instructions that decode it, about 348 per 16 keys (331 before weights had a remainder: 113 for V, 91 for K,
// 48 for the copies), with the 16 warps an SM that 128 registers leave: issue at 63 %, ALU at 53 %, no other
// unit above 40 %. A second launch, the join, costs 2 to 4 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "paged.h"
#include "sm100_ptx.cuh"

namespace sage {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxCluster = 8;  // the portable size
constexpr int kThreads = 32 * kWarps;
// Probabilities are kept as 2^shift exp2(s - m), the factor cancels in the end. fp16: 2^8, so that weights
// down to 2^-22 of the maximum keep 11 bits and the largest (2^8 2^4) is far from its limit. bf16: 2^-16, so
// that sums over values at the type's limit, which is binary32's, stay finite; when a lane's sum of weights passes
// kFull, its warp halves its sums and all further weights. A warp's eight lanes then hold at most 8 (kFull + a tile's
// 4 2^-12) of the largest value, about half. (Values at the other end, the smallest normal ones, keep more bits
// than the output has over 2^15 keys a warp.) Parts are joined as averages, whose weights add up to one.
constexpr float kSlack = 4.0f;
constexpr float kFull = 0x1p-4f;

template <typename T>
struct Is {
  static constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// Plain shared loads (ordered by the waits before them, free to move among the arithmetic).
__device__ __forceinline__ uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint2 lds64(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint32_t lds16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
__device__ __forceinline__ uint32_t lds8(const uint8_t* p) { return *p; }

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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared memory of CTA `rank` of the cluster, at the place of this CTA's `p`.
__device__ __forceinline__ uint32_t at_rank(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_cluster2(const float* p, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at_rank(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(const float* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at_rank(p, rank)) : "memory");
  return v;
}

// Weights of two heads rounded into one operand word; a and b become the rounded values.
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

// Shared memory of a CTA: per warp kStages stages of kKeys keys' K and V (FP4: codes of K, codes of
// V, scales of K, scales of V), then the meeting area of the warps.
template <int D, bool FP4>
struct Smem {
  static constexpr int kKeys = tile_keys(FP4, D) / kWarps;
  static constexpr int kKey = FP4 ? D / 2 : 2 * D;  // bytes of a key's codes or elements
  static constexpr int kSf = FP4 ? D / 16 : 0;
  static constexpr int kV = kKeys * kKey;                                 // offsets in a stage
  [[maybe_unused]] static constexpr int kKs = 2 * kV, kVs = kKs + kKeys * kSf;
  static constexpr int kStage = 2 * kKeys * (kKey + kSf);
  // Measured when chosen (us): 16-bit D = 128, 16 sequences of 256 to 16384 tokens, 8 heads: 3 stages of 16 keys and two
  // CTAs an SM 98.8, 2 stages and three CTAs 100.9. D = 64, 8 sequences of 2000 to 8192, 16 heads: 2 stages of 32
  // keys and three CTAs 39.8, 3 and two 40.9. FP4, 64 sequences of 128 to 8192: 2 stages and four CTAs 91, 3
  // and three 97, 4 and two 112; 16 keys a warp and tile 106.
  static constexpr int kStages = !FP4 && D == 128 ? 3 : 2;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMeet = kWarps * 4 * D * 4;  // four heads at a time
  static constexpr int kBytes = kRing + kMeet + kWarps * 8 * 3 * 4;
};

// Row of the V codes' stage that key `key` takes: a lane's keys 2t, 2t+1, 2t+8, 2t+9 lie in rows
// t, 4+t, 8+t, 12+t, so the four lanes of a quad read consecutive rows (with the chunk
// swizzle of D = 128, every read is free of bank conflicts).
__device__ __forceinline__ int v_row(int key) { return (key & ~7) | ((key & 1) << 2) | ((key >> 1) & 3); }

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
__device__ __forceinline__ void scores_fp4(const uint8_t* stage, int k0, int r, int t4,
                                           const uint32_t (&qf)[NT][D / 16][2], float (&s)[NT][4]) {
  using S = Smem<D, true>;
  constexpr int W = D / 32;  // code words of a lane and key: 4 or 2
  uint32_t w[2][W], sc[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int key = k0 + r + 8 * half;
    const uint8_t* sf = stage + S::kKs + key * S::kSf;
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

// O^T += V^T P^T over 16 FP4 keys, with TWO also that of pl, what the rounding of the weights left (else
// P holds both, in columns of their own). Lane (r, t4) takes channels r D/8 .. of keys 2t, 2t+1, 2t+8,
// 2t+9; the operand wants two keys' values of one channel side by side, so the nibbles of two keys are
// interleaved before they are decoded.
template <int D, int NT, bool TWO>
__device__ __forceinline__ void values_fp4(const uint8_t* stage, int k0, int r, int t4, const uint32_t (&pb)[NT][2],
                                           const uint32_t (&pl)[NT][2], float (&o)[NT][D / 16][4]) {
  using S = Smem<D, true>;
  constexpr int W = D / 64;  // code words of a lane and key: 2 or 1
  uint32_t w[4][W], sc[2];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint8_t* row = stage + S::kV + (k0 + 4 * e + t4) * S::kKey;
    if constexpr (D == 128) {
      const uint2 v = lds64(row + (((r >> 1) ^ (t4 & 2)) << 4) + (r & 1) * 8);
      w[e][0] = v.x; w[e][1] = v.y;
    } else {
      w[e][0] = lds32(row + r * 4);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* sf = stage + S::kVs + (k0 + 8 * h + 2 * t4) * S::kSf + (D == 128 ? r : r >> 1);
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
      for (int n = 0; n < NT; ++n) {
        mma16816<false>(o[n][4 * i + e], a, pb[n][0], pb[n][1]);
        if constexpr (TWO) mma16816<false>(o[n][4 * i + e], a, pl[n][0], pl[n][1]);
      }
    }
  }
}

// 1 / a sum of weights (2^-20 to 2^42), to 2 units in the last place; 0 of 0: no keys.
__device__ __forceinline__ float inverse(float sum) { return sum == 0.0f ? 0.0f : __fdividef(1.0f, sum); }

// Rounds the output, once.
template <typename T, int N>
__device__ __forceinline__ void store_out(T* out, const float (&acc)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    if constexpr (Is<T>::bf16) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * e], acc[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      w[e] = pack_half2(acc[2 * e], acc[2 * e + 1]);
    }
  }
  if constexpr (N == 8) *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (N == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(out) = w[0];
}

// What a pair costs besides its tiles (its queries, the meeting of the warps), in tiles. Measured on
// the ragged FP4 batch (us): 0 91.6, 1 84.6, 2 84.0, 3 85.8; on one long sequence 44.7, 44.9, 45.2, 45.6.
constexpr int kPairCost = 1;

// Tiles of a sequence: at least one, so that empty sequences too get their (zero) output.
template <bool FP4, int D>
__device__ __forceinline__ int tiles_of(int len) {
  return len > 0 ? (len + tile_keys(FP4, D) - 1) / tile_keys(FP4, D) : 1;
}

__device__ __forceinline__ int length_of(const CacheView& c, int b, uint32_t* err) {
  const int len = __ldg(c.lens + b);
  if (len >= 0 && len <= c.capacity) return len;
  if (err != nullptr) atomicOr(err, kDevErrSeqlens);
  return len < 0 ? 0 : c.capacity;
}

// Cost of all sequences (of one head chunk), and in `mine` of those before this thread's range of
// ceil(B / kThreads) sequences; by the whole block.
template <bool FP4, int D>
__device__ __forceinline__ int64_t count_tiles(const CacheView& c, int64_t* red, int64_t* mine, uint32_t* err) {
  const int per = (c.B + kThreads - 1) / kThreads, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int lo = min(c.B, static_cast<int>(threadIdx.x) * per), hi = min(c.B, lo + per);
  int64_t s = 0;
  for (int b = lo; b < hi; ++b) s += tiles_of<FP4, D>(length_of(c, b, err)) + kPairCost;
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

// Place in the row of tiles: sequence, key/value head, chunk of its query heads, tile; `at` counts costs from
// the share's beginning.
struct Cursor {
  int b, hk, chunk, t, len, nt, at;
};

}  // namespace

// DIRECT: a cluster of p.cluster CTAs takes one pair, each an equal part of its tiles, and joins the parts through
// distributed shared memory: no partials in global memory, no second launch.
// HT: query heads of a column tile, 8 or 4. With 4, columns 4 to 7 are the same heads once more, and take what the
// rounding of their weights leaves; with 8 that is a second product, whose operands do not fit 128 registers on FP4
// with D = 128 (64 sequences of 128 to 8192 tokens, 64 heads on 8: four CTAs an SM 92.0 us, three 89.1; D = 64, where
// they do, 57.7 and 58.7).
template <typename T, int D, int NT, int HT, bool FP4, bool DIRECT>
__global__ void __launch_bounds__(kThreads, NT == 2 ? 2 : FP4 ? (HT == 8 && D == 128 ? 3 : 4) : D == 128 ? 2 : 3)
    decode_kernel(const __grid_constant__ DecodeParams p) {
  using S = Smem<D, FP4>;
  constexpr bool kMmaBf16 = Is<T>::bf16 && !FP4;  // FP4 values are exact in fp16
  constexpr float kShift = kMmaBf16 ? -16.0f : 8.0f;
  static_assert(HT == 8 || (HT == 4 && NT == 1 && FP4));
  constexpr int KS = D / 16;                      // contraction steps of S^T, channel tiles of O^T
  constexpr int KW = S::kKeys, G = KW / 16;       // keys of a warp and tile, in groups of 16
  // All shared memory is this array: behind any static one it would begin off a 128-byte line, and the copies into
  // it then take two requests each (measured: 108 us instead of 82 for 16 sequences of 8192 tokens, 8 heads).
  extern __shared__ __align__(1024) uint8_t smem[];
  float* meet = reinterpret_cast<float*>(smem + S::kRing);
  float* meet_ml = meet + kWarps * 4 * D;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, t4 = lane & 3;
  const CacheView& c = p.c;
  const int HC = c.Hkv * p.chunks;

  wait_for_stream();
  Cursor pc;  // where the copies are
  pc.at = 0;
  int span;
  [[maybe_unused]] int64_t u0 = 0, W = 0;
  [[maybe_unused]] int shares = 0, my_share = 0;
  [[maybe_unused]] bool by_pair = false;
  if constexpr (DIRECT) {
    const int pair = blockIdx.x / p.cluster, rank = blockIdx.x - pair * p.cluster;
    const int hc = pair % HC;
    pc.b = pair / HC;
    pc.hk = hc / p.chunks;
    pc.chunk = hc - pc.hk * p.chunks;
    pc.len = length_of(c, pc.b, hc == 0 && rank == 0 && tid == 0 ? p.err : nullptr);
    pc.nt = tiles_of<FP4, D>(pc.len);
    pc.t = static_cast<int>(static_cast<int64_t>(pc.nt) * rank / p.cluster);
    span = static_cast<int>(static_cast<int64_t>(pc.nt) * (rank + 1) / p.cluster) - pc.t;
  } else {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // join_kernel may be launched: it waits for the end
    // This CTA's share, and where it begins.
    int64_t before;
    int64_t* red = reinterpret_cast<int64_t*>(meet);  // (not in use yet): per warp, then where the share begins
    int64_t& s_before = red[kWarps];
    int64_t& s_b = red[kWarps + 1];
    // p.side > 1: the shares are of one head's tiles, and p.side = HC blocks with the same share, each of its own head
    // (chunk), run side by side.
    const int stacked = p.side > 1 ? 1 : HC;
    my_share = blockIdx.x / p.side;
    W = count_tiles<FP4, D>(c, red, &before, blockIdx.x == 0 ? p.err : nullptr) * stacked;
    // Never more shares than tiles: shares of nothing between others would be loaded by the join for nothing (4
    // sequences of 3555 to 16573 FP4 tokens, one head: 12.9 us with them, 10.8 without).
    shares = static_cast<int>(min(static_cast<int64_t>(p.grid / p.side), W));
    u0 = share(W, my_share, shares);
    span = my_share < shares ? static_cast<int>(share(W, my_share + 1, shares) - u0) : 0;
    {
      const int per = (c.B + kThreads - 1) / kThreads;
      const int lo = min(c.B, tid * per), hi = min(c.B, lo + per);
      for (int b = lo; b < hi; ++b) {
        const int64_t n = tiles_of<FP4, D>(length_of(c, b, nullptr)) + kPairCost;
        if (before * stacked <= u0 && u0 < (before + n) * stacked) {
          s_b = b;
          s_before = before;
        }
        before += n;
      }
    }
    __syncthreads();
    by_pair = p.joins < p.grid;  // (see the records below)
    if (span > 0) {
      pc.b = static_cast<int>(s_b);
      pc.len = length_of(c, pc.b, nullptr);
      pc.nt = tiles_of<FP4, D>(pc.len);
      const int64_t in = u0 - s_before * stacked;
      const int above = static_cast<int>(in / (pc.nt + kPairCost));  // (0 side by side)
      const int hc = p.side > 1 ? blockIdx.x - my_share * p.side : above;
      const int rest = static_cast<int>(in - static_cast<int64_t>(above) * (pc.nt + kPairCost)) - kPairCost;
      pc.t = max(rest, 0);
      pc.at = max(-rest, 0);
      pc.hk = hc / p.chunks;
      pc.chunk = hc - pc.hk * p.chunks;
    }
    if (pc.at >= span) {  // no tile in this share (uniform over the block): a join skips it
      if (tid < 8 * NT) {
        float* ml = p.part_ml + (static_cast<int64_t>(blockIdx.x) * 2 * (8 * NT) + tid) * 2;
        ml[0] = -INFINITY;
        ml[1] = 0.0f;
      }
      if (tid == 0 && !by_pair) p.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
      return;
    }
  }
  Cursor cc = pc;  // where the arithmetic is

  auto advance = [&](Cursor& x) {
    ++x.at;
    ++x.t;
    if (DIRECT || x.t < x.nt) return;
    x.at += kPairCost;
    x.t = 0;
    if (p.side == 1) {
      if (++x.chunk < p.chunks) return;
      x.chunk = 0;
      if (++x.hk < c.Hkv) return;
      x.hk = 0;
    }
    if (++x.b < c.B) {
      x.len = length_of(c, x.b, nullptr);
      x.nt = tiles_of<FP4, D>(x.len);
    }
  };
  constexpr int KL = KW < 32 ? KW : 32, L = KW / KL;  // keys of a warp that are copied together, and how often
  const int my_key = warp * KW + lane % KL;  // of a tile (KL = 16: lanes 16 apart hold the same key), and every 32nd on
  // The page of this lane's key, loaded one tile ahead (-1: no such key, or no such page).
  auto page_of = [&](const Cursor& x, int l) -> int {
    const int pos = x.t * tile_keys(FP4, D) + my_key + 32 * l;
    if (pos >= x.len) return -1;
    const int page = __ldg(c.table + x.b * c.table_stride + div_by_page(c.page, pos));
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(c.num_pages)) {
      atomicOr(p.err, kDevErrPages);
      return -1;
    }
    return page;
  };
  const uint32_t ring = smem_u32(smem) + warp * (S::kStages * S::kStage);
  constexpr int CPK = S::kKey / 16, KPI = 32 / CPK;  // 16-byte chunks per key, keys per copy instruction
  const int ch = lane % CPK, kk = lane / CPK;
  const char* const k_src = static_cast<const char*>(c.k) + ch * 16;
  const char* const v_src = static_cast<const char*>(c.v) + ch * 16;
  const uint32_t k_at = FP4 ? kk * S::kKey + (ch << 4) : kk * S::kKey + ((ch ^ (kk & 7)) << 4);
  const uint32_t v_at = !FP4 ? k_at : v_row(kk) * S::kKey + ((D == 128 ? ch ^ (v_row(kk) & 2) : ch) << 4);
  auto copy_rows = [&](uint32_t ko, uint32_t vo, uint32_t stage, [[maybe_unused]] uint32_t sf, auto all) {
    // ALL: every key is there, so the copies need no length of their own.
    constexpr bool ALL = decltype(all)::value;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t lane_at = half ? v_at : k_at;
#pragma unroll
      for (int i = 0; i < KL / KPI; ++i) {
        const uint32_t o = __shfl_sync(0xffffffffu, half ? vo : ko, i * KPI + kk);
        const bool valid = ALL || o != 0xffffffffu;
        // 16-bit: the part of the swizzle that i brings flips chunk bits (rows are multiples of 128 bytes)
        const uint32_t at = stage + (FP4 ? lane_at : lane_at ^ (((KPI * i) & 7) << 4)) + half * S::kV + i * KPI * S::kKey;
        const char* src = (half ? v_src : k_src) + static_cast<uint64_t>(valid ? o : 0u) * 16;
        if constexpr (ALL) cp_async16(at, src);
        else cp_async16(at, src, valid);
      }
    }
    if constexpr (FP4) {
      const bool valid = ALL || ko != 0xffffffffu;
      cp_async_small<S::kSf>(sf + S::kKs + lane * S::kSf, c.k_sf + static_cast<uint64_t>(valid ? ko : 0u) * 2, valid);
      cp_async_small<S::kSf>(sf + S::kVs + lane * S::kSf, c.v_sf + static_cast<uint64_t>(valid ? vo : 0u) * 2, valid);
    }
  };
  // The same where the warp's keys lie one behind the other (consecutive slots of one page): one address, at
  // fixed distances from this lane's own key's, serves all copies of a kind. Measured (us): FP4 batch 81.2 -> 78.4,
  // one long FP4 sequence 42.7 -> 41.7; 16-bit caches, which are not bound by instructions, the same.
  auto copy_run = [&](uint32_t ko, uint32_t vo, uint32_t stage, [[maybe_unused]] uint32_t sf) {
    const int64_t back = static_cast<int64_t>(lane * 16) - (lane % KL) * S::kKey;
    const char* ks = static_cast<const char*>(c.k) + back + static_cast<uint64_t>(ko) * 16;
    const char* vs = static_cast<const char*>(c.v) + back + static_cast<uint64_t>(vo) * 16;
#pragma unroll
    for (int i = 0; i < KL / KPI; ++i) {
      const uint32_t flip = FP4 ? 0 : ((KPI * i) & 7) << 4;
      cp_async16(stage + (k_at ^ flip) + i * KPI * S::kKey, ks + i * 512);
      cp_async16(stage + S::kV + (v_at ^ flip) + i * KPI * S::kKey, vs + i * 512);
    }
    if constexpr (FP4) {
      cp_async_small<S::kSf>(sf + S::kKs + lane * S::kSf, c.k_sf + static_cast<uint64_t>(ko) * 2, true);
      cp_async_small<S::kSf>(sf + S::kVs + lane * S::kSf, c.v_sf + static_cast<uint64_t>(vo) * 2, true);
    }
  };
  int page[L];
  auto pages = [&]() {
#pragma unroll
    for (int l = 0; l < L; ++l) page[l] = page_of(pc, l);
  };
  auto copy_tile = [&](uint32_t stage) {
    if (pc.t * tile_keys(FP4, D) + warp * KW >= pc.len) return;
#pragma unroll
    for (int l = 0; l < L; ++l) {
      // This lane's key as row offsets in units of 16 bytes; all ones: no such key.
      const uint32_t pos = pc.t * tile_keys(FP4, D) + my_key + 32 * l;
      const uint32_t slot = pos - div_by_page(c.page, pos) * c.page.d;
      const uint32_t ko = page[l] * p.ku[0] + pc.hk * p.ku[1] + slot * p.ku[2];
      const uint32_t vo = page[l] * p.vu[0] + pc.hk * p.vu[1] + slot * p.vu[2];
      const uint32_t at = stage + l * KL * S::kKey, sf = stage + l * KL * S::kSf;
      if (__all_sync(0xffffffffu, page[l] >= 0)) {
        if (p.run) copy_run(ko, vo, at, sf);
        else copy_rows(ko, vo, at, sf, std::true_type{});
      } else {
        copy_rows(page[l] >= 0 ? ko : 0xffffffffu, page[l] >= 0 ? vo : 0xffffffffu, at, sf, std::false_type{});
      }
    }
  };

  if (pc.at < span) pages();
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) {
    if (pc.at < span) {
      copy_tile(ring + i * S::kStage);
      advance(pc);
      if (pc.at < span) pages();
    }
    cp_async_commit();
  }

  uint32_t qf[NT][KS][2];
  // Per head column: the running maximum m and the score that makes it rise, both unscaled: a score's difference to m is
  // taken before the scaling, so that it is exact near the maximum, however large the scores (scaled first, the step
  // of binary32 beyond 2^26 would carry the best key's weight out of its type).
  float o[NT][KS][4], m[NT][2], rise[NT][2], l[NT][2], qs[NT][2];
  [[maybe_unused]] float down = kShift;  // (bf16) the exponent of weights at the maximum
  [[maybe_unused]] const float rest = t4 < 2 ? 0.0f : 1.0f;  // (HT = 4) columns of what the rounding leaves
  uint32_t slot = 0, fill = S::kStages - 1;  // stages to read and to refill
  bool first = true;
  int head0 = pc.hk * p.group + pc.chunk * p.chunk_heads, heads = min(p.chunk_heads, p.group - pc.chunk * p.chunk_heads);
  // (DIRECT) the CTA's part for the others: outputs [8 NT][D], then (maximum, sum) per head. It takes
  // the ring's place, whose last tile has been read when the warps meet.
  [[maybe_unused]] float* part_o = reinterpret_cast<float*>(smem);
  [[maybe_unused]] float* part_ml = part_o + 8 * NT * D;
  while (cc.at < span) {
    if (first) {  // a new pair: its queries
      first = false;
      down = kShift;
      head0 = cc.hk * p.group + cc.chunk * p.chunk_heads;
      heads = min(p.chunk_heads, p.group - cc.chunk * p.chunk_heads);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int h = n * 8 + r % HT;
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
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qs[n][e] = fmaxf(p.scale_log2 * sc[e], 1.2e-38f);  // never 0: masked scores stay -inf
          m[n][e] = rise[n][e] = -FLT_MAX;                    // (finite: -inf - m stays -inf)
          l[n][e] = 0.0f;
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][s][e] = 0.0f;
      }
    }
    cp_async_wait<S::kStages - 2>();
    __syncwarp();  // this tile has arrived for every lane, and every lane has read the one before
    if (pc.at < span) {
      copy_tile(ring + fill * S::kStage);
      advance(pc);
      if (pc.at < span) pages();
    }
    cp_async_commit();
    const int k0 = cc.t * tile_keys(FP4, D) + warp * KW;
    if (k0 < cc.len) {
      const uint32_t stage = ring + slot * S::kStage;
      [[maybe_unused]] const uint8_t* stage_p = smem + warp * (S::kStages * S::kStage) + slot * S::kStage;
      float s[G][NT][4];
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[g][n][e] = 0.0f;
        if constexpr (!FP4) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int key = 16 * g + (lane & 7) + (lane & 8), c2 = 2 * k + (lane >> 4);
            uint32_t a[4];
            ldsm4(stage + key * S::kKey + ((c2 ^ (key & 7)) << 4), a);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<kMmaBf16>(s[g][n], a, qf[n][k][0], qf[n][k][1]);
          }
        } else {
          scores_fp4<D, NT>(stage_p, 16 * g, r, t4, qf, s[g]);
        }
      }
      if (k0 + KW > cc.len) {  // the sequence ends in here
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (k0 + 16 * g + (e < 2 ? 0 : 8) + r >= cc.len) s[g][n][e] = -INFINITY;
      }
      float top[NT][2];
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[n][e] = fmaxf(s[0][n][e], s[0][n][e + 2]);
#pragma unroll
          for (int g = 1; g < G; ++g) top[n][e] = fmaxf(top[n][e], fmaxf(s[g][n][e], s[g][n][e + 2]));
          raise |= top[n][e] > rise[n][e];
          if constexpr (kMmaBf16) raise |= l[n][e] > kFull;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[n][e];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x = fmaxf(x, m[n][e]);
            const float f = ex2_approx((m[n][e] - x) * qs[n][e]);
            m[n][e] = x;
            rise[n][e] = __fadd_rd(x, kSlack / qs[n][e]);
            l[n][e] *= f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[n][k][e] *= f;
              o[n][k][e + 2] *= f;
            }
          }
        if constexpr (kMmaBf16) {
          bool full = false;
#pragma unroll
          for (int n = 0; n < NT; ++n) full |= l[n][0] > kFull || l[n][1] > kFull;
          if (__any_sync(0xffffffffu, full)) {
            down -= 1.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              l[n][0] *= 0.5f;
              l[n][1] *= 0.5f;
#pragma unroll
              for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][k][e] *= 0.5f;
            }
          }
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        // Weights as operands: the rounded weight and, in an operand or columns of its own, what the rounding left,
        // rounded in turn (2^-16 of the weight in bf16, 2^-22 in fp16). One rounding alone would be as large as the
        // output's (of bf16; of fp16 on FP4 caches).
        uint32_t pb[NT][2];
        [[maybe_unused]] uint32_t pl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[g][n][e] = ex2_approx(fmaf(s[g][n][e] - m[n][e & 1], qs[n][e & 1], kMmaBf16 ? down : kShift));
          float h[4] = {s[g][n][0], s[g][n][1], s[g][n][2], s[g][n][3]};
          const uint32_t w[2] = {pack_p<kMmaBf16>(h[0], h[1]), pack_p<kMmaBf16>(h[2], h[3])};
          // (HT = 4: the weight itself in columns 0 to 3, by a factor of 0)
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = HT == 4 ? fmaf(-h[e], rest, s[g][n][e]) : s[g][n][e] - h[e];
          const uint32_t left[2] = {pack_p<kMmaBf16>(h[0], h[1]), pack_p<kMmaBf16>(h[2], h[3])};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            pb[n][e] = movm_t(HT == 4 ? left[e] : w[e]);
            if constexpr (HT == 8) pl[n][e] = movm_t(left[e]);
          }
          l[n][0] += s[g][n][0] + s[g][n][2];
          l[n][1] += s[g][n][1] + s[g][n][3];
        }
        if constexpr (!FP4) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int key = 16 * g + (lane & 7) + ((lane & 16) >> 1), c2 = 2 * k + ((lane >> 3) & 1);
            uint32_t a[4];
            ldsm4_t(stage + S::kV + key * S::kKey + ((c2 ^ (key & 7)) << 4), a);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816<kMmaBf16>(o[n][k], a, pb[n][0], pb[n][1]);
              mma16816<kMmaBf16>(o[n][k], a, pl[n][0], pl[n][1]);
            }
          }
        } else {
          values_fp4<D, NT, HT == 8>(stage_p, 16 * g, r, t4, pb, pl, o);
        }
      }
    }
    slot = slot + 1 == S::kStages ? 0 : slot + 1;
    fill = fill + 1 == S::kStages ? 0 : fill + 1;

    const Cursor at = cc;
    advance(cc);
    if ((DIRECT || at.t + 1 < at.nt) && cc.at < span) continue;
    // The pair ends, here or with this share: the warps meet.
    first = true;
    const bool begun = at.at >= at.t, whole = DIRECT ? p.cluster == 1 : begun && at.t + 1 == at.nt;
    // Partial 0: a pair that began before this share; partial 1: one that only goes on after it.
    const int part = begun ? 1 : 0;
    if (!DIRECT && tid == 0 && (by_pair ? begun : cc.at >= span)) {
      // What join_kernel has to do, one record per pair (by the CTA with the pair's first tile) or, when
      // there are more pairs than CTAs, one per CTA (for the pair that goes on after it).
      int4 rec = make_int4(-1, 0, 0, 0);
      if (begun && !whole) {
        const int64_t end = u0 + at.at - at.t + at.nt;  // past the pair's last tile
        rec = make_int4(at.b, at.hk * p.chunks + at.chunk, my_share,
                        static_cast<int>((end * shares - 1) / W));
      }
      p.rec[by_pair ? static_cast<int64_t>(at.b) * HC + at.hk * p.chunks + at.chunk : blockIdx.x] = rec;
    }
    if constexpr (HT == 4) {  // columns 0 to 3 get the sums of both
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][k][e] += __shfl_xor_sync(0xffffffffu, o[0][k][e], 2);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
      }
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {  // heads 0-3, then 4-7
        if (n * 8 + pass * 4 >= heads) break;  // uniform over the block
        __syncthreads();                       // the area's last readers are done
        if (r == 0 && pass == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // scaled, for the joining; -inf: no keys
            float* ml = meet_ml + (warp * 8 + 2 * t4 + e) * 3;
            ml[0] = l[n][e] == 0.0f ? -INFINITY : fmaxf(m[n][e] * qs[n][e], -FLT_MAX);
            ml[1] = l[n][e];
            ml[2] = kMmaBf16 ? __int_as_float((127 + static_cast<int>(kShift - down)) << 23) : 1.0f;  // what halving took
          }
        }
        if ((t4 >> 1) == pass) {
          float* row = meet + (warp * 4 + 2 * (t4 & 1)) * D;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            // Channels of a tile's two rows: neighbours of the lane's own range in FP4, else 8 apart.
            const int ch = FP4 ? (D / 8) * r + 2 * k : 16 * k + r;
            constexpr int step = FP4 ? 1 : 8;
            row[ch] = o[n][k][0];
            row[D + ch] = o[n][k][1];
            row[ch + step] = o[n][k][2];
            row[D + ch + step] = o[n][k][3];
          }
        }
        __syncthreads();
        // 32 threads per head, D / 32 channels each.
        constexpr int N = D / 32;
        const int hh = tid >> 5, h = pass * 4 + hh, c0 = (tid & 31) * N;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, meet_ml[(w * 8 + h) * 3]);
        float acc[N], sum = 0.0f, wt[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* ml = meet_ml + (w * 8 + h) * 3;
          wt[w] = ml[0] == -INFINITY ? 0.0f : ml[2] * ex2_approx(ml[0] - mx);
          sum += ml[1] * wt[w];
        }
        const float inv = inverse(sum);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = wt[w] * inv;
          const float2* src = reinterpret_cast<const float2*>(meet + (w * 4 + hh) * D + c0);
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            acc[e] += src[e / 2].x * f;
            acc[e + 1] += src[e / 2].y * f;
          }
        }
        if (n * 8 + h < heads) {
          if (whole) {
            T* out = static_cast<T*>(p.out) + at.b * p.sob + static_cast<int64_t>(head0 + n * 8 + h) * p.soh + c0;
            store_out<T, N>(out, acc);
          } else if constexpr (DIRECT) {
            float2* po = reinterpret_cast<float2*>(part_o + (n * 8 + h) * D + c0);
#pragma unroll
            for (int e = 0; e < N; e += 2) po[e / 2] = make_float2(acc[e], acc[e + 1]);
            if ((tid & 31) == 0) {
              part_ml[(n * 8 + h) * 2] = mx;
              part_ml[(n * 8 + h) * 2 + 1] = sum;
            }
          } else {
            const int64_t g = (static_cast<int64_t>(blockIdx.x) * 2 + part) * (8 * NT) + n * 8 + h;
            float2* po = reinterpret_cast<float2*>(p.part_o + g * D + c0);
#pragma unroll
            for (int e = 0; e < N; e += 2) po[e / 2] = make_float2(acc[e], acc[e + 1]);
            if ((tid & 31) == 0) {
              p.part_ml[g * 2] = mx;
              p.part_ml[g * 2 + 1] = sum;
            }
          }
        }
      }
    }
  }
  if constexpr (DIRECT) {
    if (p.cluster == 1) return;  // uniform over the grid
    if (span <= 0 && tid < 8 * NT) {  // no tile here, no output
      part_ml[2 * tid] = -INFINITY;
      part_ml[2 * tid + 1] = 0.0f;
    }
    cluster_sync();
    constexpr int Q = D / 4;  // a thread's piece: 4 channels of a head
    const int rank = blockIdx.x % p.cluster;
    for (int i = rank * kThreads + tid; i < heads * Q; i += p.cluster * kThreads) {
      const int h = i / Q, c0 = (i - h * Q) * 4;
      float2 ml[kMaxCluster];
      float4 v[kMaxCluster];
      float mx = -INFINITY;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        ml[r] = make_float2(-INFINITY, 0.0f);
        if (r < p.cluster) {
          ml[r] = ld_cluster2(part_ml + 2 * h, r);
          if (ml[r].x != -INFINITY) v[r] = ld_cluster4(part_o + h * D + c0, r);
        }
        mx = fmaxf(mx, ml[r].x);
      }
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (ml[r].x != -INFINITY) ml[r].y *= ex2_approx(ml[r].x - mx);
        sum += ml[r].y;
      }
      const float inv = inverse(sum);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (ml[r].x == -INFINITY) continue;
        const float f = ml[r].y * inv;
        acc[0] += v[r].x * f;
        acc[1] += v[r].y * f;
        acc[2] += v[r].z * f;
        acc[3] += v[r].w * f;
      }
      store_out<T, 4>(static_cast<T*>(p.out) + pc.b * p.sob + static_cast<int64_t>(head0 + h) * p.soh + c0, acc);
    }
    cluster_sync();  // the parts stay until every CTA has read them
  }
}

// Adds up the partial results of the pairs that lie in more than one share. Block (record, head); its G groups
// of 16 threads take every G-th share each, then meet. G is 16 where there are few pairs (each in many shares), else
// 8: the blocks wait on the machine for the shares to end, and larger ones are in their way (us, G = 8 / 16 / 32:
// one sequence of 131071 FP4 tokens 41.7 / 40.5 / 40.8, ragged FP4 batch 78.5 / 81.9 / 97.5).
constexpr int kMaxGroups = 16;

template <typename T, int D, int NT>
__global__ void __launch_bounds__(16 * kMaxGroups) join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int N = D / 16;
  __shared__ float s_acc[kMaxGroups][D];
  __shared__ float s_ml[kMaxGroups][2];
  const int tid = threadIdx.x, G = blockDim.x >> 4, g = tid >> 4, c0 = (tid & 15) * N, h = blockIdx.y;
  wait_for_stream();
  const int4 rec = p.rec[blockIdx.x];
  if (rec.x < 0) return;
  const int hk = rec.y / p.chunks, chunk = rec.y - hk * p.chunks;
  if (h >= min(p.chunk_heads, p.group - chunk * p.chunk_heads)) return;
  auto row_of = [&](int share) {
    const int cta = p.side > 1 ? share * p.side + rec.y : share;
    return (static_cast<int64_t>(cta) * 2 + (share == rec.z ? 1 : 0)) * (8 * NT) + h;
  };
  float mx = -INFINITY, acc[N], sum = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.0f;
  constexpr int U = 4;  // partials loaded together, before their maxima are known
  for (int first = rec.z + g; first <= rec.w; first += G * U) {
    float m[U], l[U];
    float4 v[U][N / 4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[u] = -INFINITY;
      l[u] = 0.0f;
      if (first + G * u <= rec.w) {
        const int64_t row = row_of(first + G * u);
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + row * 2);
        m[u] = ml.x;
        l[u] = ml.y;
#pragma unroll
        for (int e = 0; e < N / 4; ++e) v[u][e] = *reinterpret_cast<const float4*>(p.part_o + row * D + c0 + 4 * e);
      }
    }
    // The average so far and the new ones, each by its share of the weights.
    float top = mx;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, m[u]);
    if (top == -INFINITY) continue;  // empty shares
    float f0 = mx == -INFINITY ? 0.0f : sum * ex2_approx(mx - top);
    mx = top;
    sum = f0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      l[u] *= m[u] == -INFINITY ? 0.0f : ex2_approx(m[u] - top);
      sum += l[u];
    }
    const float inv = inverse(sum);
    f0 *= inv;
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] *= f0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (m[u] == -INFINITY) continue;  // none, or an empty share, which has no output
      const float f = l[u] * inv;
#pragma unroll
      for (int e = 0; e < N / 4; ++e) {
        acc[4 * e] += v[u][e].x * f;
        acc[4 * e + 1] += v[u][e].y * f;
        acc[4 * e + 2] += v[u][e].z * f;
        acc[4 * e + 3] += v[u][e].w * f;
      }
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
  // The groups' averages by their shares of the weights: thread i (of 16) forms group i's.
  const float m = tid < G ? s_ml[tid][0] : -INFINITY;
  float wt = tid < G ? s_ml[tid][1] : 0.0f;
  mx = m;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffu, mx, o));
  wt = m == -INFINITY ? 0.0f : wt * ex2_approx(m - mx);
  sum = wt;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffu, sum, o);
  wt *= inverse(sum);
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.0f;
#pragma unroll 8
  for (int i = 0; i < G; ++i) {
    const float f = __shfl_sync(0xffffu, wt, i);
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] += s_acc[i][c0 + e] * f;
  }
  const int64_t head = static_cast<int64_t>(hk) * p.group + chunk * p.chunk_heads + h;
  store_out<T, N>(static_cast<T*>(p.out) + rec.x * p.sob + head * p.soh + c0, acc);
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

template <typename T, int D, int NT, int HT, bool FP4>
cudaError_t launch_one(DecodeParams p, int max_grid, cudaStream_t stream) {
  constexpr int smem = Smem<D, FP4>::kBytes;
  p.run = p.c.sk.n == D && p.c.sv.n == D && p.c.page.d % (Smem<D, FP4>::kKeys < 32 ? Smem<D, FP4>::kKeys : 32) == 0;
  cudaError_t e = cudaSuccess;
  const int fit = resident_ctas<decode_kernel<T, D, NT, HT, FP4, false>>(smem, &e);
  if (e != cudaSuccess) return e;
  const int64_t pairs = static_cast<int64_t>(p.c.B) * p.c.Hkv * p.chunks;
  const int tiles = p.c.capacity > 0 ? (p.c.capacity - 1) / tile_keys(FP4, D) + 1 : 1;
  int cluster = 1;
  while (cluster < kMaxCluster && cluster < tiles && pairs * cluster * 2 <= fit) cluster *= 2;
  // One launch by pairs where a CTA then has few tiles: at most 8 (lengths may be ragged, and nothing evens
  // them out), and no more than three above its share of all tiles, which is about what the second launch
  // costs; with far more pairs than CTAs the shares' pipeline across pairs wins. Measured by pairs / by
  // shares (us, sequences x tokens, 32 heads on 8, D 128): 16-bit, 1 x 64 3.7 / 4.6, 1 x 1024 6.8 / 6.9,
  // 1 x 4096 11.3 / 9.3, 4 x 2048 9.8 / 10.7, 16 x 512 8.9 / 11.2, 16 x 1024 16.4 / 18.3, 16 x 1024 to 8192
  // 63 / 48, 64 x 512 27.2 / 29.7, 200 x 64 22.5 / 19.4; FP4, 1 x 1024 6.7 / 7.8, 16 x 4096 24.3 / 26.8,
  // 64 x 1024 23.0 / 28.7, 64 x 256 to 2048 35.0 / 32.4, 200 x 512 34.4 / 42.6 (when chosen).
  const int per = (tiles + cluster - 1) / cluster;
  if (pairs <= 3 * static_cast<int64_t>(fit) && per <= 8 && per <= pairs * (tiles + 1) / fit + 3) {
    resident_ctas<decode_kernel<T, D, NT, HT, FP4, true>>(smem, &e);
    if (e != cudaSuccess) return e;
    p.cluster = cluster;
    return launch_dependent(decode_kernel<T, D, NT, HT, FP4, true>, dim3(static_cast<unsigned>(pairs * cluster)), kThreads,
                            smem, stream, p, cluster);
  }
  p.grid = max_grid < fit ? max_grid : fit;
  const int HC = p.c.Hkv * p.chunks, groups = p.grid / HC;
  p.side = 1;
  // Shares of one head each, the heads side by side: their blocks read the same tokens' rows at the same time, so that
  // a token's rows of all heads (adjacent in NHD order, where a head's 32 bytes of codes and 4 of scales are
  // parts of the DRAM's and L2's units) and the page table are fetched once. It needs a multiple of HC blocks, and the
  // rest of the machine stays idle: up to an eighth of it in NHD order, almost nothing otherwise. Measured by
  // all heads' tiles end to end / side by side (us): FP4, 10 sequences of 24078 to 78702 tokens, 56 heads on 8, D = 64
  // NHD 218.6 / 109.7 (end to end it read 3.9 times its bytes from DRAM), HND 109.6 / 107.6, D = 128 NHD 231 / 177,
  // HND 165.4 / 166.9; 16 sequences of 256 to 16384, 32 heads on 8: FP4 D = 64 NHD 34.7 / 30.1, HND 28.0 / 27.5,
  // D = 128 NHD 47.2 / 43.0, HND 41.0 / 40.3, 16-bit D = 64 NHD 48.9 / 44.3, HND 44.7 / 43.7, D = 128 NHD 82.3 /
  // 80.9, HND 84.4 / 81.6. It loses a little where head-major pages share nothing and the shares come out less even:
  // besides the D = 128 HND case above, 16-bit, 16 sequences of 128 to 8192, 64 heads on 4, HND 34.3 / 35.2.
  const bool nhd = p.c.sk.h < p.c.sk.n && p.c.sv.h < p.c.sv.n;
  if (groups * HC * 64 >= p.grid * (nhd ? 56 : 63)) {
    p.side = HC;
    p.grid = groups * HC;
  }
  p.joins = static_cast<int>(pairs < p.grid ? pairs : p.grid);
  e = launch_dependent(decode_kernel<T, D, NT, HT, FP4, false>, dim3(p.grid), kThreads, smem, stream, p);
  if (e != cudaSuccess || p.c.capacity <= tile_keys(FP4, D)) return e;  // one tile per pair: none is split
  const bool few = static_cast<int64_t>(p.joins) * p.chunk_heads <= 148;
  return launch_dependent(join_kernel<T, D, NT>, dim3(p.joins, p.chunk_heads), few ? 16 * kMaxGroups : 128, 0, stream, p);
}

// FP4 caches with at most four heads a chunk: every head in two columns, so that the remainders of the weights
// cost no product of their own. Measured, two columns / two products (us): FP4, 64 sequences of 128 to 8192
// tokens, 32 heads on 8, D 128 80.0 / 88.1, D 64 52.0 / 55.9; one sequence of 131071 41.2 / 45.1. 16-bit caches
// are not bound by the products.
template <typename T, int D>
cudaError_t launch_format(const DecodeParams& p, bool fp4, int NT, int max_grid, cudaStream_t stream) {
  if (!fp4)
    return NT == 1 ? launch_one<T, D, 1, 8, false>(p, max_grid, stream) : launch_one<T, D, 2, 8, false>(p, max_grid, stream);
  if (p.chunk_heads <= 4) return launch_one<T, D, 1, 4, true>(p, max_grid, stream);
  return NT == 1 ? launch_one<T, D, 1, 8, true>(p, max_grid, stream) : launch_one<T, D, 2, 8, true>(p, max_grid, stream);
}

template <typename T>
cudaError_t launch_type(const DecodeParams& p, int D, bool fp4, int NT, int max_grid, cudaStream_t stream) {
  return D == 128 ? launch_format<T, 128>(p, fp4, NT, max_grid, stream) : launch_format<T, 64>(p, fp4, NT, max_grid, stream);
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& p, int D, int dtype, bool fp4, int NT, int max_grid, cudaStream_t stream) {
  return dtype == kDtypeBF16 ? launch_type<__nv_bfloat16>(p, D, fp4, NT, max_grid, stream)
                             : launch_type<__half>(p, D, fp4, NT, max_grid, stream);
}

}  // namespace sage
