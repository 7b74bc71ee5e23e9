// Row kernels of the paged cache (sm_100a): norm and rotation of query / key heads, the same
// with keys and values going into cache pages, and reading pages back.
//
// One head of one token is a row of D channels. D / 16 lanes own a row, two 8-channel chunks each, as far
// apart as the two halves of a rotation pair (i, i + R/2): neither pairing needs a shuffle, and
// neighbouring lanes move neighbouring chunks; only the mean square and the FP4 block maximum cross
// lanes. A lane group keeps its token's cosines, sines and norm weights in registers over the heads of its
// item; the arithmetic runs on two channels per instruction. Each row is read once and written once: the
// floor of all three is HBM. Measured on several B200s, share of the 6549 GB/s a copy reaches: norm and
// rotation of B1 H24 N32768 D128 144 to 148 us, 5.6 to 5.7 TB/s (0.85 to 0.87); prompt of 8191 tokens, 32 + 8
// heads, 31.4 us, 5.4 TB/s (0.83); dense read of 123,171 cached FP4 tokens, 8 heads, 107 us, 6.04 TB/s (0.92).
// Append of 17,823 tokens, 8 key/value heads, 16-bit 30.3 us (0.74), FP4 41.3 us (0.35), with 32 query heads
// 90.5 (0.74) and 87.7 (0.67): nothing is saturated there (issue at 34 % and 47 %, ALU 25 % and 33 %). 128
// registers leave 16 warps an SM (19 % of its warps active) to hide a chain of loads to a token's place, the
// rows' own latency and, for FP4, the reductions and conversions of the encoding.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "fp4_encode.cuh"
#include "paged.h"
#include "sm100_ptx.cuh"

namespace sage {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack(uint4 raw, float* x) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    r = *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    r = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float* x) {
  return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// Eight norm weights from channel c on.
template <typename T>
__device__ __forceinline__ void load_weights(const void* w, int w32, int c, float* x) {
  if (w32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
    const float4 a = __ldg(f), b = __ldg(f + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    unpack<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(w) + c)), x);
  }
}

// 16 channels as eight pairs (a, b): pair i is (i, i + 8), or (2i, 2i + 1) when interleaved.
template <bool INTER>
__device__ __forceinline__ void split(const float (&x)[16], float2 (&a)[4], float2 (&b)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = INTER ? make_float2(x[4 * i], x[4 * i + 2]) : make_float2(x[2 * i], x[2 * i + 1]);
    b[i] = INTER ? make_float2(x[4 * i + 1], x[4 * i + 3]) : make_float2(x[2 * i + 8], x[2 * i + 9]);
  }
}
template <bool INTER>
__device__ __forceinline__ void join(const float2 (&a)[4], const float2 (&b)[4], float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[INTER ? 4 * i : 2 * i] = a[i].x;
    x[INTER ? 4 * i + 2 : 2 * i + 1] = a[i].y;
    x[INTER ? 4 * i + 1 : 2 * i + 8] = b[i].x;
    x[INTER ? 4 * i + 3 : 2 * i + 9] = b[i].y;
  }
}

// RN32(1 / sqrt(m)) of a binary64 m: the binary32 estimate refined by two Newton steps in
// binary64 (each squares the relative error, ~2^-22 at first), so that the result is the
// correctly rounded one up to the rare value within ~2^-50 of a rounding border. m far outside
// binary32's range is brought into it by an even power of two.
// Rows so small (subnormals) that the inverse would leave binary32 are scaled up on the way.
__device__ __forceinline__ float rsqrt_exact(double m, float2 (&xa)[4], float2 (&xb)[4]) {
  if (m < 1e-70 && m > 0.0) {
    const float2 up = make_float2(0x1p64f, 0x1p64f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xa[i] = mul2(xa[i], up);
      xb[i] = mul2(xb[i], up);
    }
    m *= 0x1p128;
  }
  double back = 1.0;
  if (m < 1e-36) {
    m *= 0x1p160;
    back = 0x1p80;
  } else if (m > 1e37) {
    m *= 0x1p-200;
    back = 0x1p-100;
  }
  const float f = rsqrtf(static_cast<float>(m));
  if (!(f > 0.0f && f < INFINITY)) return f;  // of 0, infinity, NaN
  double y = static_cast<double>(f);
  const double h = 0.5 * m;
  y = y * fma(-h * y, y, 1.5);
  y = y * fma(-h * y, y, 1.5);
  return static_cast<float>(y * back);
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Largest magnitude of x[O .. O + 7]; NaN if one of them is.
template <int O>
__device__ __forceinline__ float absmax8(const float (&x)[16]) {
  float a = max3_nan(fabsf(x[O]), fabsf(x[O + 1]), fabsf(x[O + 2]));
  a = max3_nan(a, fabsf(x[O + 3]), fabsf(x[O + 4]));
  a = max3_nan(a, fabsf(x[O + 5]), fabsf(x[O + 6]));
  return max3_nan(a, fabsf(x[O + 7]), 0.0f);
}

// Where a token of an append or gather call lies in the cache.
struct Place {
  int64_t page;  // -1: nowhere (outside the sequences, or refused and reported)
  int slot, pos;
};

__device__ __forceinline__ Place place_of(const CacheView& c, int tok, bool lead, uint32_t* err) {
  Place r{-1, 0, 0};
  int b = tok, first = tok, n = 1;
  if (c.cu != nullptr) {
    int lo = 0, hi = c.B;  // the last b with cu[b] <= tok
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(c.cu + mid) <= tok) lo = mid;
      else hi = mid;
    }
    b = lo;
    first = __ldg(c.cu + b);
    const int end = __ldg(c.cu + b + 1);
    n = end - first;
    // Rows behind the last sequence; before the first, or a negative offset (with which the differences below
    // could leave 32 bits): a bad table.
    if (first < 0 || tok < first || tok >= end) {
      if ((first < 0 || tok < first) && lead) atomicOr(err, kDevErrSeqlens);
      return r;
    }
  } else if (b >= c.B) {
    return r;
  }
  const int len = __ldg(c.lens + b);
  const int64_t pos = static_cast<int64_t>(len) - n + (tok - first);
  if (pos < 0 || len > c.capacity) {
    if (lead) atomicOr(err, kDevErrSeqlens);
    return r;
  }
  r.pos = static_cast<int>(pos);
  const uint32_t i = div_by_page(c.page, r.pos);
  r.slot = r.pos - static_cast<int>(i * c.page.d);
  const int page = __ldg(c.table + static_cast<int64_t>(b) * c.table_stride + i);
  if (page < 0 || page >= c.num_pages) {
    if (lead) atomicOr(err, kDevErrPages);
    return r;
  }
  r.page = page;
  return r;
}

}  // namespace

// Item (token group, head range of one set): a warp holds 32 / (D / 16) tokens and walks the
// heads. CACHE: keys and values go to their pages (FP4: quantized), else keys to dense rows.
// INTER: rotation pairs are adjacent channels.
//
// Rows in flight per lane group: four loaded together, or two with the next two already on their way
// where the arithmetic of quantization has to be hidden. Measured (us, 128 registers, 16 warps an
// SM): norm and interleaved rotation of B1 H24 N32768 D128 143 against 143, prompt of 8191 tokens with 32 + 8
// heads 31.8 against 35.6, append of 17,823 tokens to an FP4 cache and its read 131 against 115 (when chosen). Three
// blocks' worth of registers (80) spill and lose a quarter; 8 channels a lane need as many instructions
// for half the bytes and lose 40 %.
template <typename T, int D, bool CACHE, bool FP4, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int LPR = D / 16, GPW = 32 / LPR;
  constexpr int kUnroll = FP4 ? 2 : 4;
  constexpr bool kAhead = FP4;
  wait_for_stream();
  const int lane = threadIdx.x & 31, j = lane % LPR;
  const int items = p.items_q + p.items_k + p.items_v;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  const int64_t tg = w / items;
  int it = static_cast<int>(w - tg * items);
  if (tg * GPW >= p.T) return;
  const int64_t tok = tg * GPW + lane / LPR;
  bool ok = tok < p.T;
  // The item's set of heads.
  int set = 0, H = p.Hq, per = p.per_q;
  if (it >= p.items_q) {
    it -= p.items_q;
    set = 1;
    H = p.Hk;
    per = p.per_k;
    if (it >= p.items_k) {
      it -= p.items_k;
      set = 2;
      H = p.Hv;
      per = p.per_v;
    }
  }
  const int h0 = it * per, h1 = min(H, h0 + per);
  const char* src = static_cast<const char*>(set == 0 ? p.q : set == 1 ? p.k : p.v);
  const Strides ss = set == 0 ? p.sq : set == 1 ? p.sk : p.sv;

  // The token's place and position.
  Place at{-1, 0, 0};
  int64_t b = 0, n = tok;
  if (ok) {
    if constexpr (CACHE) {
      at = place_of(p.c, static_cast<int>(tok), j == 0, p.err);
      ok = at.page >= 0;
    } else {
      b = tok / p.N;
      n = tok - b * p.N;
      at.pos = p.positions != nullptr ? __ldg(p.positions + tok) : static_cast<int>(n);
    }
    if (ok && p.rope != nullptr && (at.pos < 0 || at.pos >= p.rope_len)) {
      if (j == 0) atomicOr(p.err, kDevErrSeqlens);
      ok = false;
    }
  }
  const int R = set == 2 || p.rope == nullptr ? 0 : p.R;
  const int half = R / 16;
  const bool rot = j < half;
  // The lane's chunks: two as far apart as the halves of the rotated channels, or of the others, so that
  // neighbouring lanes read and write neighbouring chunks (adjacent pairs per lane fetch every sector twice).
  const int ca = rot ? j : R / 16 + j, cb = rot ? j + half : ca + D / 16 - half;

  // Cosines and sines of the lane's eight pairs, two to a register pair.
  float2 cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = make_float2(1.0f, 1.0f);
    sn[i] = make_float2(0.0f, 0.0f);
  }
  if (ok && rot) {
    const float* row = p.rope + static_cast<int64_t>(at.pos) * R;
    const int oa = INTER ? 4 * ca : 8 * ca, ob = INTER ? 4 * cb : 8 * ca + 4;
    const float* cos_sin[2] = {row, row + R / 2};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(cos_sin[k] + oa));
      const float4 b4 = __ldg(reinterpret_cast<const float4*>(cos_sin[k] + ob));
      float2* to = k == 0 ? cs : sn;
      to[0] = make_float2(a.x, a.y);
      to[1] = make_float2(a.z, a.w);
      to[2] = make_float2(b4.x, b4.y);
      to[3] = make_float2(b4.z, b4.w);
    }
  }
  const void* wp = set == 0 ? p.qw : set == 1 ? p.kw : nullptr;
  float2 wa[4], wb[4];
  if (wp != nullptr) {
    float t[16];
    load_weights<T>(wp, p.w32, 8 * ca, t);
    load_weights<T>(wp, p.w32, 8 * cb, t + 8);
    split<INTER>(t, wa, wb);
  }

  const bool paged = CACHE && set != 0;
  const Strides ds = paged ? (set == 1 ? p.c.sk : p.c.sv) : (set == 0 ? p.sqo : p.sko);
  const int64_t dst_tok = paged ? at.page * ds.b + at.slot * ds.n : b * ds.b + n * ds.n;
  char* dst = static_cast<char*>(paged ? (set == 1 ? p.c.k : p.c.v) : set == 0 ? p.qo : p.ko);
  uint8_t* sf = set == 1 ? p.c.k_sf : p.c.v_sf;
  const char* row_a = src + (b * ss.b + n * ss.n) * 2 + ca * 16;
  const int to_b = (cb - ca) * 16;

  uint4 raw[kUnroll][2];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
      if (ok && h + u < h1) {
        const char* row = row_a + static_cast<int64_t>(h + u) * ss.h * 2;
        raw[u][0] = ld_stream(row);
        raw[u][1] = ld_stream(row + to_b);
      }
    }
  };
  load(h0);
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 now[kUnroll][2];
    if (!kAhead && h != h0) load(h);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      now[u][0] = raw[u][0];
      now[u][1] = raw[u][1];
    }
    if (kAhead) load(h + kUnroll);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= h1) break;  // uniform over the warp
      const int64_t row = dst_tok + static_cast<int64_t>(h + u) * ds.h;
      if (!(FP4 && paged) && wp == nullptr && R == 0) {
        if (ok) {
          *reinterpret_cast<uint4*>(dst + row * 2 + ca * 16) = now[u][0];
          *reinterpret_cast<uint4*>(dst + row * 2 + cb * 16) = now[u][1];
        }
        continue;
      }
      // Pair i of the lane: (xa, xb), eight of them.
      float2 xa[4], xb[4];
      {
        float t[16];
        unpack<T>(now[u][0], t);
        unpack<T>(now[u][1], t + 8);
        split<INTER>(t, xa, xb);
      }
      if (wp != nullptr) {
        float r;
        if (FP4 && paged) {
          // 4-bit codes depend on the last bit: the mean square in binary64, where the order of the
          // sum does not matter (squares of 16-bit values are exact there).
          double s2[2] = {0.0, 0.0};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s2[0] = fma(static_cast<double>(xa[i].x), static_cast<double>(xa[i].x), s2[0]);
            s2[1] = fma(static_cast<double>(xa[i].y), static_cast<double>(xa[i].y), s2[1]);
            s2[0] = fma(static_cast<double>(xb[i].x), static_cast<double>(xb[i].x), s2[0]);
            s2[1] = fma(static_cast<double>(xb[i].y), static_cast<double>(xb[i].y), s2[1]);
          }
          double s = s2[0] + s2[1];
#pragma unroll
          for (int o = 1; o < LPR; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          r = rsqrt_exact(s * (1.0 / D) + static_cast<double>(p.eps), xa, xb);
        } else {
          float2 s2 = make_float2(0.0f, 0.0f), t2 = s2;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s2 = fma2(xa[i], xa[i], s2);
            t2 = fma2(xb[i], xb[i], t2);
          }
          s2 = add2(s2, t2);
          float s = s2.x + s2.y;
#pragma unroll
          for (int o = 1; o < LPR; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          s = s * (1.0f / D) + p.eps;
          r = rsqrtf(s);
          if (!(s > 1e-30f && s < 1e37f)) {  // squares beyond binary32's range (uniform over the row's lanes)
            double m = 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              m += static_cast<double>(xa[i].x) * xa[i].x + static_cast<double>(xa[i].y) * xa[i].y;
              m += static_cast<double>(xb[i].x) * xb[i].x + static_cast<double>(xb[i].y) * xb[i].y;
            }
            const uint32_t group = (LPR == 8 ? 0xffu : 0xfu) << (lane & ~(LPR - 1));
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) m += __shfl_xor_sync(group, m, o);
            r = rsqrt_exact(m * (1.0 / D) + static_cast<double>(p.eps), xa, xb);
          }
        }
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xa[i] = mul2(mul2(xa[i], r2), wa[i]);
          xb[i] = mul2(mul2(xb[i], r2), wb[i]);
        }
      }
      if (rot) {
        // Products and sums each rounded on their own (no fused multiply-add), as a chain of
        // elementwise operations rounds them: codes then agree bit for bit. A mul.rn.f32x2 is contracted with
        // the sum behind it (243 of two million fp16 outputs differ), a fused product with a -0 that only
        // the host knows is not, and rounds the same.
        const float2 mz = make_float2(p.minus_zero, p.minus_zero);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = xa[i], c = xb[i];
          xa[i] = sub2(fma2(a, cs[i], mz), fma2(c, sn[i], mz));
          xb[i] = add2(fma2(c, cs[i], mz), fma2(a, sn[i], mz));
        }
      }
      float x[16];  // channels of the two chunks in order
      join<INTER>(xa, xb, x);
      if (FP4 && paged) {
        float ma = absmax8<0>(x), mb = absmax8<8>(x);
        if (!(fmaxf(ma, mb) < INFINITY) || ma != ma || mb != mb) {  // saturate (NaN: to the largest)
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = fmaxf(fminf(x[i], FLT_MAX), -FLT_MAX);
          ma = absmax8<0>(x);
          mb = absmax8<8>(x);
        }
        // A block is two neighbouring chunks, one each of lanes j and j ^ 1.
        const uint32_t ba = block_scale_byte(fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 1)));
        const uint32_t bb = block_scale_byte(fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 1)));
        const uint32_t ea = encode8_neg<0>(x, e4m3_to_f32(ba)), eb = encode8_neg<8>(x, e4m3_to_f32(bb));
        if (ok) {
          char* codes = dst + row / 2;
          uint8_t* scales = sf + row / 16;
          *reinterpret_cast<uint32_t*>(codes + 4 * ca) = ea;
          *reinterpret_cast<uint32_t*>(codes + 4 * cb) = eb;
          if ((j & 1) == 0) {
            scales[ca / 2] = static_cast<uint8_t>(ba);
            scales[cb / 2] = static_cast<uint8_t>(bb);
          }
        }
      } else if (ok) {
        *reinterpret_cast<uint4*>(dst + row * 2 + ca * 16) = pack<T>(x);
        *reinterpret_cast<uint4*>(dst + row * 2 + cb * 16) = pack<T>(x + 8);
      }
    }
  }
}

// Item (token group, head range of K or of V): rows of the cache to dense rows.
template <typename T, int D, bool FP4>
__global__ void __launch_bounds__(kThreads, 4) gather_kernel(const GatherParams p) {
  constexpr int LPR = D / 16, GPW = 32 / LPR, kUnroll = 4;
  wait_for_stream();
  const int lane = threadIdx.x & 31, j = lane % LPR;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  const int64_t tg = w / (2 * p.items);
  int it = static_cast<int>(w - tg * (2 * p.items));
  if (tg * GPW >= p.T) return;
  const int64_t tok = tg * GPW + lane / LPR;
  if (tok >= p.T) return;  // no shuffles below
  const bool is_v = it >= p.items;
  if (is_v) it -= p.items;
  const int h0 = it * p.heads_per_item, h1 = min(p.c.Hkv, h0 + p.heads_per_item);
  const Place at = place_of(p.c, static_cast<int>(tok), j == 0, p.err);
  if (at.page < 0) return;
  const Strides ss = is_v ? p.c.sv : p.c.sk, ds = is_v ? p.sv : p.sk;
  const char* src = static_cast<const char*>(is_v ? p.c.v : p.c.k);
  const uint8_t* sf = is_v ? p.c.v_sf : p.c.k_sf;
  // The lane's two chunks of 8 channels are D / 2 apart: neighbouring lanes write neighbouring chunks.
  char* dst = static_cast<char*>(is_v ? p.v : p.k) + (tok * ds.n + 8 * j) * 2;
  const int64_t src_tok = at.page * ss.b + at.slot * ss.n;
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 raw[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= h1) continue;
      const int64_t row = src_tok + static_cast<int64_t>(h + u) * ss.h;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (FP4) {
          raw[u][i].x = *reinterpret_cast<const uint32_t*>(src + row / 2 + 4 * j + i * (D / 4));
          raw[u][i].y = sf[row / 16 + j / 2 + i * (D / 32)];
        } else {
          raw[u][i] = ld_stream(src + row * 2 + 16 * j + i * D);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= h1) continue;
      char* row = dst + static_cast<int64_t>(h + u) * ds.h * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (FP4) {
          // E2M1 times E4M3 has at most six significant bits and fits fp16's range: every product
          // below is exact, in fp16 and after it in bf16.
          const float sc = e4m3_to_f32(raw[u][i].y);
          const __half2 s2 = __floats2half2_rn(sc, sc);
          uint32_t v[4], o[4];
          e2m1x8_to_f16x2(raw[u][i].x, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 m = __hmul2(*reinterpret_cast<const __half2*>(&v[e]), s2);
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
              const float2 f = __half22float2(m);
              o[e] = pack2<T>(f.x, f.y);
            } else {
              o[e] = *reinterpret_cast<const uint32_t*>(&m);
            }
          }
          raw[u][i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        *reinterpret_cast<uint4*>(row + i * D) = raw[u][i];
      }
    }
  }
}

template <typename T, int D, bool INTER>
static cudaError_t rows_of(const RowsParams& p, bool to_cache, bool fp4, unsigned grid, cudaStream_t stream) {
  auto* kernel = !to_cache ? rows_kernel<T, D, false, false, INTER>
                 : fp4     ? rows_kernel<T, D, true, true, INTER>
                           : rows_kernel<T, D, true, false, INTER>;
  return launch_dependent(kernel, dim3(grid), kThreads, 0, stream, p);
}

template <typename T>
static cudaError_t rows_of_type(const RowsParams& p, int D, bool to_cache, bool fp4, unsigned grid,
                                cudaStream_t stream) {
  if (D == 128)
    return p.interleaved ? rows_of<T, 128, true>(p, to_cache, fp4, grid, stream)
                         : rows_of<T, 128, false>(p, to_cache, fp4, grid, stream);
  return p.interleaved ? rows_of<T, 64, true>(p, to_cache, fp4, grid, stream)
                       : rows_of<T, 64, false>(p, to_cache, fp4, grid, stream);
}

// Heads a warp walks: as many as leave `waves` times the warps that are resident (148 SMs of 16), at
// most 16. Dense rows: four times (with one, the prompt above takes 32.7 us instead of 31.3). Paged ones: once, as
// finding a token's place is a chain of loads (with four, keys and values of 17,823 tokens, 8 heads, took 48.4 us
// instead of 41.5 to FP4 pages and 35.1 instead of 31.8 to 16-bit ones).
static int heads_of(int64_t groups, int heads, int waves) {
  int n = 16;
  while (n > 1 && groups * ((heads + n - 1) / n) < waves * 148 * 16) n /= 2;
  return n;
}

cudaError_t launch_rows(const RowsParams& in, int D, int dtype, bool to_cache, bool fp4, cudaStream_t stream) {
  RowsParams p = in;
  p.minus_zero = -0.0f;
  const int gpw = 512 / D;
  const int64_t groups = (static_cast<int64_t>(p.T) + gpw - 1) / gpw;
  const int most = heads_of(groups, p.Hq + p.Hk + p.Hv, to_cache ? 1 : 4);
  auto split = [&](int h, int* items, int* per) {
    *items = (h + most - 1) / most;
    *per = h > 0 ? (h + *items - 1) / *items : 0;
  };
  split(p.Hq, &p.items_q, &p.per_q);
  split(p.Hk, &p.items_k, &p.per_k);
  split(p.Hv, &p.items_v, &p.per_v);
  const int64_t warps = groups * (p.items_q + p.items_k + p.items_v);
  const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  return dtype == kDtypeBF16 ? rows_of_type<__nv_bfloat16>(p, D, to_cache, fp4, grid, stream)
                             : rows_of_type<__half>(p, D, to_cache, fp4, grid, stream);
}

template <typename T, int D>
static cudaError_t gather_of(const GatherParams& p, bool fp4, unsigned grid, cudaStream_t stream) {
  return launch_dependent(fp4 ? gather_kernel<T, D, true> : gather_kernel<T, D, false>, dim3(grid), kThreads, 0, stream, p);
}

cudaError_t launch_gather(const GatherParams& in, int D, int dtype, bool fp4, cudaStream_t stream) {
  GatherParams p = in;
  const int gpw = 512 / D;
  const int64_t groups = (static_cast<int64_t>(p.T) + gpw - 1) / gpw;
  p.heads_per_item = heads_of(groups, 2 * p.c.Hkv, 1);
  p.items = (p.c.Hkv + p.heads_per_item - 1) / p.heads_per_item;
  const int64_t warps = groups * 2 * p.items;
  const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (dtype == kDtypeBF16)
    return D == 128 ? gather_of<__nv_bfloat16, 128>(p, fp4, grid, stream) : gather_of<__nv_bfloat16, 64>(p, fp4, grid, stream);
  return D == 128 ? gather_of<__half, 128>(p, fp4, grid, stream) : gather_of<__half, 64>(p, fp4, grid, stream);
}

}  // namespace sage
