// Microscaled 4-bit floating point: rows of e2m1 values under block scales, and their
// product on the tensor cores (tcgen05.mma kind::mxf4nvf4, fp32 accumulate).
//
// Formats.  Elements are e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, packed
// two to a byte with the even column in the low half.
//   MXFP4  blocks of 32 columns, scale 2^(c - 127) stored as the byte c (e8m0)
//   NVFP4  blocks of 16 columns, scale an e4m3 byte, and one fp32 scale per row
// Block scales are stored as the tensor core takes them: tiles of 128 rows x 4 blocks,
// 512 bytes each, tiles row-major; row i, block j of a tile is byte
// (i % 32) * 16 + (i / 32) * 4 + j.  Blocks outside the matrix hold zero.
#pragma once
#include <cuda_fp4.h>

#include "zi_attention.cuh"  // packed fp32 pairs
#include "zi_cluster.cuh"
#include "zi_common.cuh"
#include "zi_gemm.cuh"

namespace zi {
namespace fp4 {

enum : int { MX = 0, NV = 1 };

template <int FMT>
constexpr int kBlock = FMT == MX ? 32 : 16;

constexpr int kTileBytes = 512;  // one scale tile: 128 rows x 4 blocks

// Scale tiles along a row of `cols` columns / down `rows` rows.
template <int FMT>
__host__ __device__ constexpr int tiles_along(int cols) {
  return (cols + 4 * kBlock<FMT> - 1) / (4 * kBlock<FMT>);
}
__host__ __device__ constexpr int tiles_down(int rows) { return (rows + 127) / 128; }

// Offset of the 4-byte word that holds the scales of `row`'s blocks 4 tile .. 4 tile + 3.
ZI_DEV size_t scale_word(int row, int tile, int tiles_x) {
  return (size_t(row >> 7) * tiles_x + tile) * kTileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// ------------------------------------------------------------------ rows

constexpr int kRowsThreads = 256;
constexpr int kRowsMaxCols = 16384;  // four spans of 16 columns on each thread of a CTA

// From this many rows on the rows alone fill the GPU, and fewer threads per row with more loads on their way each are
// faster.  Measured with one and four 32-byte spans per thread: 20480 x 3840 bf16 to NVFP4 62.7 / 46.6 us, 4128 x
// 3840 14.8 / 12.3.
constexpr int kDeepRows = 1024;

// How quantize_kernel takes rows of `cols` columns: threads per row, a power of two that is at least the threads of one
// scale word, and spans per thread (1 to kMaxSpans, each compiled).  tpr * spans >= cols / 16.
struct RowsPlan {
  int tpr, spans;
};
constexpr int kMaxSpans = 4;
__host__ inline RowsPlan rows_plan(int rows, int cols, int bytes) {
  const int all = cols / 16;
  auto each = [&](int tpr) { return (all + tpr - 1) / tpr; };
  int tpr = 8;
  while (tpr < all && tpr < kRowsThreads) tpr *= 2;
  // fp32 spans are twice as long: two of them are as many loads.  Three spans become five or six with half the threads;
  // those counts, compiled too, were slower up to 4,128 rows or up to 8% faster past that (1024 x 1536 bf16 to NVFP4 4.0
  // against 3.1 us, 20480 x 10240 100 against 108), and three run as four took 4128 x 10240 from 25.3 to 27.8
  const int deep = bytes == 4 ? 2 : 4;
  while (rows >= kDeepRows && each(tpr) < deep && tpr > 8 && each(tpr / 2) <= kMaxSpans) tpr /= 2;
  return {tpr, each(tpr)};
}
static_assert(kRowsMaxCols / 16 <= kMaxSpans * kRowsThreads, "spans per thread");

// 16 consecutive elements of a row, as loaded.
template <typename TIn>
struct Span {
  uint4 w[sizeof(TIn)];  // 2 or 4 of 16 bytes
};

template <typename TIn>
ZI_DEV Span<TIn> load_span(const TIn* p) {
  Span<TIn> s;
#pragma unroll
  for (int i = 0; i < int(sizeof(TIn)); ++i) s.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return s;
}

// The largest |x| as its bit pattern (an integer maximum, so that infinities and NaN come out
// on top instead of being dropped).
ZI_DEV uint32_t span_amax(const Span<float>& s) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = max(m, max(max(s.w[i].x & 0x7FFFFFFFu, s.w[i].y & 0x7FFFFFFFu), max(s.w[i].z & 0x7FFFFFFFu, s.w[i].w & 0x7FFFFFFFu)));
  return m;
}
ZI_DEV uint32_t span_amax(const Span<uint16_t>& s) {
  uint32_t m = 0;  // two 16-bit maxima
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m = __vmaxu2(m, __vmaxu2(s.w[i].x & 0x7FFF7FFFu, s.w[i].y & 0x7FFF7FFFu));
    m = __vmaxu2(m, __vmaxu2(s.w[i].z & 0x7FFF7FFFu, s.w[i].w & 0x7FFF7FFFu));
  }
  return max(m << 16, m & 0xFFFF0000u);
}

ZI_DEV void span_values(const Span<float>& s, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[4 * i] = __uint_as_float(s.w[i].x);
    v[4 * i + 1] = __uint_as_float(s.w[i].y);
    v[4 * i + 2] = __uint_as_float(s.w[i].z);
    v[4 * i + 3] = __uint_as_float(s.w[i].w);
  }
}
ZI_DEV void span_values(const Span<uint16_t>& s, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t b[4] = {s.w[i].x, s.w[i].y, s.w[i].z, s.w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[8 * i + 2 * k] = __uint_as_float(b[k] << 16);
      v[8 * i + 2 * k + 1] = __uint_as_float(b[k] & 0xFFFF0000u);
    }
  }
}

ZI_DEV float rcp_approx(float x) {  // within 2^-22 or so
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr uint32_t kInfBits = 0x7F800000u;

// e8m0 byte of an MXFP4 block: floor(log2 amax) - 2 (6 = 1.5 * 2^2 is the largest
// element), at least -127; a block of zeros gets scale 1, one with an infinity or a NaN
// the NaN scale.
ZI_DEV uint32_t mx_scale(uint32_t amax) {
  if (amax >= kInfBits) return 0xFFu;
  if (amax == 0) return 127u;
  const uint32_t e = amax >> 23;  // floor(log2 amax) + 127, or 0 below the normal numbers
  return e < 2 ? 0u : e - 2;
}

// Row scale of NVFP4 as a biased exponent: the smallest power of two r with amax <= 448 *
// 6 * r (2688 = 1.3125 * 2^11), at least 2^-126; a row of zeros gets r = 1.  With a power
// of two every later product by r is exact, so the codes are those of exact arithmetic.
ZI_DEV uint32_t nv_row_exp(uint32_t amax) {
  if (amax == 0) return 127u;
  const int e = int(amax >> 23) - 11 + ((amax & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return e < 1 ? 1u : uint32_t(e);
}

ZI_DEV float exp_float(uint32_t biased) { return __uint_as_float(biased << 23); }

// q is the quotient of a by b rounded to fp32.  The borders between two e4m3 (or e2m1)
// values have at most five significant bits; when q falls on such a number the exact
// quotient may lie on either side of it, and the sign of a - q b (exact) moves q one step
// that way, so that rounding q decides as rounding the exact quotient would.
ZI_DEV float off_border(float q, float a, float b) {
  const uint32_t u = __float_as_uint(q);
  if ((u & 0x7FFFFu) == 0u) {
    const float rem = fmaf(-q, b, a);
    if (rem != 0.f && q != 0.f) return __uint_as_float((rem > 0.f) == (q > 0.f) ? u + 1 : u - 1);
  }
  return q;
}

// e4m3 byte of an NVFP4 block: amax / (6 r), rounded to nearest even.  A bf16 amax (8 bits) over 6
// is a border between two e4m3 values exactly or at least 2^-8 of its value away from it, so
// rounding the approximate quotient to fp16 first (11 bits) lands on the border if and only
// if the exact quotient does.  For an fp32 amax the remainder decides.
template <bool EXACT24>
ZI_DEV uint32_t nv_scale(uint32_t amax, uint32_t row_exp) {
  if (amax >= kInfBits) return 0x7Fu;
  const float t = __uint_as_float(amax) * exp_float(254u - row_exp);  // amax / r, exact
  const float q0 = t * (1.f / 6.f);
  if (!EXACT24) return __nv_cvt_halfraw_to_fp8(__half_raw(__float2half_rn(q0)), __NV_SATFINITE, __NV_E4M3);
  const float q = off_border(fmaf(fmaf(-q0, 6.f, t), 1.f / 6.f, q0), t, 6.f);  // one Newton step on the residual
  return __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

ZI_DEV float e4m3_float(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(byte), __NV_E4M3);
  return __half2float(__half(h));
}

// 16 e2m1 codes (8 bytes, in column order) of v, to nearest even, saturating at 6.
ZI_DEV uint2 codes16(const float* v) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w[h])
        : "f"(v[8 * h]), "f"(v[8 * h + 1]), "f"(v[8 * h + 2]), "f"(v[8 * h + 3]), "f"(v[8 * h + 4]), "f"(v[8 * h + 5]),
          "f"(v[8 * h + 6]), "f"(v[8 * h + 7]));
  return make_uint2(w[0], w[1]);
}

// v[i] to v[i] / (sc r), an NVFP4 block's elements in units of its scales, such that e2m1's rounding of it
// decides as on the exact quotient.  x times a reciprocal is off by 2^-23 or so, enough to miss a tie; adding and
// taking off 48 rounds it to a multiple of 2^-18 in the same FMA (quotients are below 9.1, and within 2^-19 of the
// exact ones before).  The ties 0.25, 0.75, ... 5 are such multiples, so a quotient lands on one only from near it:
// - a bf16 x (8 bits) over a scale of 4 bits is a tie exactly or at least 2^-8 of its value away from it;
// - an fp32 x can be that near: a span with a quotient on a multiple of 1/4 (one span in 4000) is done again by a
//   division whose remainder says on which side of the tie it lies.
template <bool EXACT24>
ZI_DEV void nv_units(float* v, float sc, uint32_t row_exp) {
  float inv = rcp_approx(sc);
  if (row_exp < 28u) {  // 1 / r would take the factor out of range: tiny rows, scaled first
    const float rinv = exp_float(254u - row_exp);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] *= rinv;
    row_exp = 127u;
  } else {
    inv *= exp_float(254u - row_exp);
  }
  constexpr float kSnap = 48.f;
  const uint64_t inv2 = f2_pack(inv, inv), up = f2_pack(kSnap, kSnap), down = f2_pack(-kSnap, -kSnap);
  float w[16];
  uint32_t low = ~0u;
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const uint64_t at = f2_fma(f2_pack(v[e], v[e + 1]), inv2, up);
    if (EXACT24) low = min(low, min(uint32_t(at) << 16, uint32_t(at >> 32) << 16));
    f2_unpack(f2_add(at, down), w[e], w[e + 1]);
  }
  if (EXACT24 && low == 0u) {
    const float rinv = exp_float(254u - row_exp), i1 = rcp_approx(sc);
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // 4 h + e without indexing the registers: the loop rotates them
        const float xr = v[e] * rinv, v0 = xr * i1;
        const float v1 = fmaf(fmaf(-v0, sc, xr), i1, v0);  // one Newton step on the residual
        const float r = copysignf(off_border(v1, xr, sc), xr);
        v[e] = v[e + 4];
        v[e + 4] = v[e + 8];
        v[e + 8] = v[e + 12];
        v[e + 12] = r;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = copysignf(w[e], v[e]);  // the sign of a zero is kept
  }
}

// Rows of x [rows, cols] to codes, block scales and (NVFP4) row scales.  `tpr` threads (a
// power of two, up to the whole CTA) per row, NB spans of 16 columns per thread, span i on
// thread i % tpr.  x is read once, all of a thread's spans at once, and an NVFP4 row waits
// in registers, as it was loaded, for its maximum.  Rows past the end up to the scale tile's
// 128 only write their zero scales.
// Bound by HBM for MXFP4 (20480 x 3840 bf16 32.2 us, 6.1 TB/s), by issue slots for NVFP4, whose rows wait for their
// maximum and whose ties are exact (same rows 40.5 us, 5.0 TB/s; 4128 x 3840 11.8 us, 4128 x 10240 24.6 us).
template <int FMT, typename TIn, int NB>
__global__ void __launch_bounds__(kRowsThreads) quantize_kernel(const TIn* __restrict__ x, int rows, int cols, int tpr,
                                                               uint8_t* __restrict__ q, uint8_t* __restrict__ bs,
                                                               float* __restrict__ rs) {
  __shared__ uint32_t red[kRowsThreads / 32];
  const int sub = threadIdx.x & (tpr - 1);
  const int row = int(blockIdx.x * (kRowsThreads / tpr) + threadIdx.x / tpr);
  const int spans = cols / 16;
  const int tiles_x = tiles_along<FMT>(cols);
  const int rows_pad = tiles_down(rows) * 128;

  Span<TIn> s[NB];
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int i = sub + k * tpr;
    if (row < rows && i < spans) {
      s[k] = load_span(x + size_t(row) * cols + size_t(i) * 16);
    } else {
#pragma unroll
      for (int e = 0; e < int(sizeof(TIn)); ++e) s[k].w[e] = make_uint4(0, 0, 0, 0);
    }
  }
  uint32_t top[NB];  // the spans' largest |x|
#pragma unroll
  for (int k = 0; k < NB; ++k) top[k] = span_amax(s[k]);
  uint32_t row_exp = 127u;
  if constexpr (FMT == NV) {
    uint32_t am = 0;
#pragma unroll
    for (int k = 0; k < NB; ++k)
      if (top[k] < kInfBits) am = max(am, top[k]);
    for (int o = (tpr < 32 ? tpr : 32) >> 1; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (tpr > 32) {  // the row spans warps
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = am;
      __syncthreads();
      const int w0 = (threadIdx.x / tpr) * (tpr / 32);
      for (int w = 0; w < tpr / 32; ++w) am = max(am, red[w0 + w]);
    }
    row_exp = nv_row_exp(am);
    if (sub == 0 && row < rows) rs[row] = exp_float(row_exp);
  }
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int i = sub + k * tpr;
    const bool have = row < rows && i < spans;
    uint32_t amax = top[k];
    if (FMT == MX) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    uint32_t byte = 0;
    if (have) {
      float v[16];
      span_values(s[k], v);
      if constexpr (FMT == MX) {
        byte = mx_scale(amax);
        const uint64_t inv2 = f2_pack(exp_float(254u - byte), exp_float(254u - byte));
#pragma unroll
        for (int e = 0; e < 16; e += 2)  // exact (a power of two), or far below half a step
          f2_unpack(f2_mul(f2_pack(v[e], v[e + 1]), inv2), v[e], v[e + 1]);
      } else {
        byte = nv_scale<sizeof(TIn) == 4>(amax, row_exp);
        if (byte != 0u && byte != 0x7Fu) {
          nv_units<sizeof(TIn) == 4>(v, e4m3_float(byte), row_exp);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = copysignf(0.f, v[e]);
        }
      }
      uint2 c = codes16(v);
      if (amax >= kInfBits) c = make_uint2(0, 0);
      *reinterpret_cast<uint2*>(q + size_t(row) * (cols / 2) + size_t(i) * 8) = c;
    }
    // four block scales to a word
    constexpr int kStep = kBlock<FMT> / 16;  // threads per block
    uint32_t word = byte;
#pragma unroll
    for (int j = 1; j < 4; ++j) word |= __shfl_down_sync(0xffffffffu, byte, j * kStep) << (8 * j);
    const int tile = i / (4 * kStep);
    if ((i & (4 * kStep - 1)) == 0 && tile < tiles_x && row < rows_pad)
      *reinterpret_cast<uint32_t*>(bs + scale_word(row, tile, tiles_x)) = word;
  }
}

// The values that codes and scales stand for, bf16 or fp32.  `tpr` threads per row, 8 columns
// (one 16- or 32-byte store) per thread at a time, so that a warp's stores are contiguous.
// Bound by its writes, small calls by their launch (20480 x 3840 MXFP4 to bf16 35 us, 5.7 TB/s; 4128 x 3840 7.2 us).
template <int FMT, typename TOut>
__global__ void __launch_bounds__(kRowsThreads) dequantize_kernel(const uint8_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ bs,
                                                                 const float* __restrict__ rs, int rows, int cols,
                                                                 int tpr, TOut* __restrict__ y) {
  const int sub = threadIdx.x & (tpr - 1);
  const int row = int(blockIdx.x * (kRowsThreads / tpr) + threadIdx.x / tpr);
  if (row >= rows) return;
  const int eights = cols / 8, tiles_x = tiles_along<FMT>(cols);
  const float r = FMT == NV ? __ldg(rs + row) : 1.f;
  const uint8_t* scales = bs + scale_word(row, 0, tiles_x);
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(q + size_t(row) * (cols / 2));
  TOut* out = y + size_t(row) * cols;
#pragma unroll 4
  for (int i = sub; i < eights; i += tpr) {
    const int block = i * 8 / kBlock<FMT>;
    const uint32_t byte = __ldg(scales + (block >> 2) * kTileBytes + (block & 3));
    const uint32_t w = __ldg(codes + i);
    float sc;
    if constexpr (FMT == MX) {
      // 2^(c - 127): c = 0 lies below the normal numbers, c = 255 is NaN
      sc = byte == 0xFFu ? __uint_as_float(0x7FC00000u) : byte == 0 ? __uint_as_float(0x00400000u) : exp_float(byte);
    } else {
      sc = e4m3_float(byte) * r;
    }
    const uint64_t sc2 = f2_pack(sc, sc);
    float v[8];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const __half2_raw c = __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t((w >> (8 * b)) & 0xFFu), __NV_E2M1);
      const float2 f = __half22float2(__half2(c));
      f2_unpack(f2_mul(f2_pack(f.x, f.y), sc2), v[2 * b], v[2 * b + 1]);
    }
    if constexpr (sizeof(TOut) == 4) {
      float4* d = reinterpret_cast<float4*>(out + size_t(i) * 8);
      d[0] = make_float4(v[0], v[1], v[2], v[3]);
      d[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(out + size_t(i) * 8) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
  }
}

// ------------------------------------------------------------------ product: shared parts

// D[tmem] (+)= (A * SA)(B * SB)^T for 64 columns of K, both operands e2m1 in smem, block
// scales in TMEM (one byte per row and block; MXFP4 2 blocks, NVFP4 4 blocks per instruction).
template <int FMT>
ZI_DEV void mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa_tmem, uint32_t sb_tmem,
                uint32_t accumulate) {
  if constexpr (FMT == MX) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
        : "memory");
  }
}

// Instruction descriptor: e2m1 A and B (format code 1), K-major, block scales e8m0 or e4m3.
// `pair`: which half of the 4-byte scale word an MXFP4 instruction takes (0 or 1).
template <int FMT>
__host__ __device__ constexpr uint32_t idesc(int M, int N, int pair) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | ((FMT == MX ? 1u : 0u) << 23) |
         (static_cast<uint32_t>(M >> 7) << 27) | (static_cast<uint32_t>(2 * pair) << 4) |
         (static_cast<uint32_t>(2 * pair) << 29);
}

// Descriptor of one 512-byte scale tile in smem for tcgen05.cp 32x128b: 32 rows of 16 bytes,
// no swizzle, 8-row groups 128 bytes apart.
ZI_DEV uint64_t scale_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128u >> 4) << 32;
  d |= 1ull << 46;
  return d;
}

// One scale tile to 4 TMEM columns (column c: rows 32 c .. 32 c + 31 on the lanes, repeated
// in every lane quarter).  Runs in order with the MMAs issued by the same thread.
ZI_DEV void copy_scales(uint32_t tmem_col, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem_col), "l"(scale_desc(saddr)) : "memory");
}

// x ra rb.  Row scales go from 2^-126 to 2^117, and two small ones multiplied with each other could give 0 and two large
// ones infinity (NaN for x = 0) where the result is in range.  Such a pair lies on one side of 1 and is taken one after
// the other: x ra then leaves the range only where the result does.
ZI_DEV float by_row_scales(float x, float ra, float rb) {
  const float both = ra * rb;
  const bool in = fabsf(both) >= 0x1p-126f && fabsf(both) <= 0x1.fffffep127f;
  const float first = in ? both : ra, second = in ? 1.f : rb;  // chosen rather than branched
  return x * first * second;
}

// Untiled bulk copy into this CTA's smem, completing on `bar`.
ZI_DEV void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem_dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

constexpr int kStageK = 256;  // columns of K per stage: 128 bytes of codes per row
template <int FMT>
constexpr int kStageTiles = kStageK / (4 * kBlock<FMT>);  // scale tiles per stage and 128 rows: 2 or 4

struct GemmParams {
  const uint8_t* abs;  // block scales of A [M, K] ...
  const uint8_t* bbs;  // ... and of B [N, K]
  const float* ars;    // row scales (NVFP4) [M], or null
  const float* brs;    // [N], or null
  uint16_t* out;       // bf16 [M, N]
  int M, N, K;
};

// ------------------------------------------------------------------ product: few rows
// One CTA per 128 rows of B (output columns) x TN rows of A (one tile of 16, 32 or 64 rows, or any number of 128: a tile's
// block scales start where a scale tile of 128 rows does), with B as the instruction's
// M operand: a call with few rows is bound by reading B, so B's rows fill the tensor core
// and A's few rows are its N.  A cluster of CTAs shares a tile's K: each takes a run of
// stages, leaves its fp32 partial in its own smem, and sums a part of the tile over the
// cluster's CTAs in rank order.  Warps: 0 loads, 1 MMA, 2..5 epilogue.
// About 6 us are fixed (launch, filling the ring, the join): 1 x 3840 x 3840 NVFP4 7.9 us against 1.3 of reading B.
// 77 x 11520 x 3840 MXFP4 14.7 us against 3.9: 90 tiles in clusters of two are 180 CTAs, so that 32 SMs hold two and the
// others one, and 77 rows run as 128.
constexpr int kNarrowThreads = 192;

template <int FMT, int TN>
struct NarrowSmem {
  static constexpr uint32_t kB = 128 * 128;                       // B: 128 rows x 128 bytes
  static constexpr uint32_t kA = TN * 128 < 1024 ? 1024 : TN * 128;
  static constexpr uint32_t kSc = kStageTiles<FMT> * kTileBytes;  // scales of one operand
  static constexpr uint32_t kStage = kB + kA + 2 * kSc;
  static constexpr int kStages = TN <= 32 ? 4 : 3;              // two CTAs per SM
  static constexpr uint32_t kBar = kStages * kStage;
  static constexpr uint32_t kBytes = kBar + 256 + 1024;
  static constexpr uint32_t kCols = TN <= 32 ? 128 : 256;         // TMEM: D, then two scale buffers
  static constexpr uint32_t kColScale = TN < 32 ? 32 : TN;
  static constexpr uint32_t kScaleCols = 2 * 4 * kStageTiles<FMT>;  // B's and A's, per buffer
  static_assert(kColScale + 2 * kScaleCols <= kCols, "TMEM columns");
  static_assert(kStage % 1024 == 0 && 128 * TN * 4 <= kBar, "stage alignment; the partial fits the ring");
  static_assert(2 * (kBytes + 1024) <= 233472, "two CTAs per SM");
};

template <int FMT, int TN>
__global__ void __launch_bounds__(kNarrowThreads)
    gemm_narrow_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, GemmParams p,
                       int splits) {
  using L = NarrowSmem<FMT, TN>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + kStages;
  uint64_t* done = empty + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(blockIdx.x) % splits;
  const int n0 = int(blockIdx.x) / splits * 128, m0 = int(blockIdx.y) * TN;
  const int stages = (p.K + kStageK - 1) / kStageK;
  const int k0 = int(static_cast<long long>(rank) * stages / splits);
  const int k1 = int(static_cast<long long>(rank + 1) * stages / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = device_error_set() ? 1 : 0;  // an earlier kernel timed out: leave everything untouched
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool skip = *abort_flag != 0;
  const int tiles_x = tiles_along<FMT>(p.K);
  const int nk = k1 - k0;

  if (!skip && warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (; it < nk; ++it) {
        const int s = it % kStages;
        if (!mbar_wait(&empty[s], ((it / kStages) & 1) ^ 1, abort_flag, ZI_DEVERR_TIMEOUT_PRODUCER)) {
          ok = false;
          break;
        }
        const int kb = k0 + it;
        const int t0 = kb * kStageTiles<FMT>;
        const uint32_t sc = uint32_t(min(kStageTiles<FMT>, tiles_x - t0)) * kTileBytes;
        uint8_t* sb = smem + s * L::kStage;
        mbar_arrive_expect_tx(&full[s], L::kB + TN * 128 + 2 * sc);
        tma_load_2d(sb, &tmB, &full[s], kb * 128, n0);
        tma_load_2d(sb + L::kB, &tmA, &full[s], kb * 128, m0);
        bulk_load(sb + L::kB + L::kA, p.bbs + (size_t(n0 >> 7) * tiles_x + t0) * kTileBytes, sc, &full[s]);
        bulk_load(sb + L::kB + L::kA + L::kSc, p.abs + (size_t(m0 >> 7) * tiles_x + t0) * kTileBytes, sc, &full[s]);
      }
      if (!ok) {  // let the copies already issued land
        volatile int never = 0;
        for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
          mbar_wait(&full[j % kStages], (j / kStages) & 1, &never, ZI_DEVERR_TIMEOUT_DRAIN);
      }
    }
  } else if (!skip && warp == 1) {
    if (lane == 0) {
      for (int it = 0; it < nk; ++it) {
        const int s = it % kStages;
        if (!mbar_wait(&full[s], (it / kStages) & 1, abort_flag, ZI_DEVERR_TIMEOUT_MMA)) break;
        tc_fence_after();
        const uint32_t b_addr = smem_u32(smem + s * L::kStage), a_addr = b_addr + L::kB, sc_addr = a_addr + L::kA;
        const uint32_t tsb = tmem + L::kColScale + (it & 1) * L::kScaleCols, tsa = tsb + 4 * kStageTiles<FMT>;
        const int kleft = p.K - (k0 + it) * kStageK;
        const int ksteps = kleft >= kStageK ? 4 : (kleft + 63) / 64;
        const int tiles = min(kStageTiles<FMT>, tiles_x - (k0 + it) * kStageTiles<FMT>);
        for (int t = 0; t < tiles; ++t) {
          copy_scales(tsb + 4 * t, sc_addr + t * kTileBytes);
          copy_scales(tsa + 4 * t, sc_addr + L::kSc + t * kTileBytes);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < ksteps) {
            const int t = FMT == MX ? k >> 1 : k;
            mma<FMT>(tmem, smem_desc_sw128(b_addr + k * 32, 16), smem_desc_sw128(a_addr + k * 32, 16),
                     idesc<FMT>(128, TN, FMT == MX ? k & 1 : 0), tsb + 4 * t, tsa + 4 * t,
                     (it | k) != 0 ? 1u : 0u);
          }
        }
        tc_commit(&empty[s]);
      }
      tc_commit(done);  // after an abort too: TMEM and smem are reused once every MMA issued has finished
      volatile int never = 0;
      mbar_wait(done, 0, &never, ZI_DEVERR_TIMEOUT_DRAIN);
    }
  }
  // the partial, column-major: [TN][128] fp32 over the ring (every copy has landed, every MMA is done)
  __syncthreads();
  tc_fence_after();
  float* part = reinterpret_cast<float*>(smem);
  const int q = warp & 3;
  if (warp >= 2 && !*abort_flag) {
#pragma unroll 1
    for (int c = 0; c < TN; c += 16) {
      uint32_t v[16];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
          "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
          : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
            "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
          : "r"(tmem + (uint32_t(q * 32) << 16) + c));
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        asm volatile("" : "+r"(v[i]));
        part[(c + i) * 128 + q * 32 + lane] = nk > 0 ? __uint_as_float(v[i]) : 0.f;
      }
    }
  }
  if (splits > 1) cluster_sync(); else __syncthreads();
  // this CTA's share of the tile's rows of A, summed over the ranks in order: a warp per row, 4 columns of the output
  // per thread, two rows at a time
  const bool bad = splits > 1 ? any_peer_set(abort_flag, splits) : *abort_flag != 0;
  const int c0 = rank * TN / splits, c1 = min((rank + 1) * TN / splits, p.M - m0);
  const int n = n0 + 4 * lane;
  if (!bad && n < p.N) {  // N is a multiple of 8
    uint32_t peer[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      peer[r] = splits > 1 ? peer_addr(smem_u32(part) + 16 * lane, r < splits ? r : 0) : smem_u32(part) + 16 * lane;
    float4 rb = make_float4(1.f, 1.f, 1.f, 1.f);
    if constexpr (FMT == NV) rb = __ldg(reinterpret_cast<const float4*>(p.brs + n));
    constexpr int kWarps = kNarrowThreads / 32;
    for (int c = c0 + warp; c < c1; c += 2 * kWarps) {
      float4 v[2][kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        v[0][r] = ld_peer4(peer[r] + c * 512, r < splits);
        v[1][r] = ld_peer4(peer[r] + (c + kWarps) * 512, r < splits && c + kWarps < c1);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int m = m0 + c + u * kWarps;
        if (c + u * kWarps < c1) {
          float4 x = v[u][0];
#pragma unroll
          for (int r = 1; r < kMaxCluster; ++r)
            if (r < splits) x = make_float4(x.x + v[u][r].x, x.y + v[u][r].y, x.z + v[u][r].z, x.w + v[u][r].w);
          if constexpr (FMT == NV) {
            const float ra = __ldg(p.ars + m);
            x = make_float4(by_row_scales(x.x, ra, rb.x), by_row_scales(x.y, ra, rb.y), by_row_scales(x.z, ra, rb.z),
                            by_row_scales(x.w, ra, rb.w));
          }
          *reinterpret_cast<uint2*>(p.out + size_t(m) * p.N + n) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
        }
      }
    }
  }
  if (splits > 1) cluster_sync(); else __syncthreads();  // no CTA leaves while its partial may be read
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// ------------------------------------------------------------------ product: many rows
// CTA pairs (cta_group::2) on 256 x 256 tiles, as gemm_pair_body: each CTA stages its own 128
// rows of A and of B (128 bytes, 256 columns, of K per stage) and the block scales that its
// tensor core needs, A's for its own rows and B's for all 256 columns; CTA 0 issues
// M = 256 MMAs for both SMs.
// - Scales reach TMEM through registers: four warps, one per lane quarter, read a stage's
//   scale tiles from smem and store them with tcgen05.st while earlier MMAs run.  tcgen05.cp
//   would do it in the tensor core's own queue, between the MMAs (4128 x 20480 x 3840 NVFP4:
//   252 us with it, 174 without when that was changed).
// - TMEM holds one accumulator (256 columns) and one scale buffer per smem stage; there is no
//   room for a second accumulator, so the epilogue warps take the whole accumulator into
//   registers (128 columns each) and hand it back before they scale and store: the MMAs of
//   the next tile wait for the TMEM reads alone.
// 4128 x 20480 x 3840: NVFP4 162 us (4.0 PFLOP/s), MXFP4 146 us (4.4).  What bounds it is not settled: the tensor pipe is
// active 54% of the time, issue slots 25%, DRAM 12%.
// Warps: 0 loads, 1 MMA, 2..3 idle, 4..7 scales, 8..15 epilogue; registers move from the
// first two warpgroups to the epilogue (128 a thread at launch; 56 + 64 + 2 x 192 = 504 <= 512).
constexpr int kWideThreads = 512;
constexpr int kWideRegsLow = 56, kWideRegsScale = 64, kWideRegsEpi = 192;

template <int FMT>
struct WideSmem {
  static constexpr uint32_t kA = 128 * 128, kB = 128 * 128;
  static constexpr uint32_t kSc = kStageTiles<FMT> * kTileBytes;  // 128 rows of scales
  static constexpr uint32_t kStage = kA + kB + 3 * kSc;
  static constexpr int kStages = 5;
  static constexpr uint32_t kOut = kStages * kStage;  // 4 KB per epilogue warp
  static constexpr uint32_t kBar = kOut + 8 * 4096;
  static constexpr uint32_t kBytes = kBar + 256 + 1024;
  static constexpr uint32_t kColScale = 256;
  static constexpr uint32_t kScaleCols = 12 * kStageTiles<FMT>;  // A's 4 and B's 8 columns per scale tile
  static_assert(kStage % 1024 == 0 && kBytes <= 232448, "stage alignment, shared memory");
  static_assert(kColScale + kStages * kScaleCols <= 512, "TMEM columns");
};

ZI_DEV void load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// As mma, over the pair: each CTA's scales come from its own TMEM.
template <int FMT>
ZI_DEV void mma2(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa_tmem, uint32_t sb_tmem,
                 uint32_t accumulate) {
  if constexpr (FMT == MX) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
        : "memory");
  }
}

// 4 consecutive columns of this warp's 32 lanes.
ZI_DEV void tmem_st4(uint32_t taddr, uint4 w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(w.x), "r"(w.y),
               "r"(w.z), "r"(w.w)
               : "memory");
}

// Whether every product of a row scale of A and one of B is in range for the whole warp, so that its epilogue need not
// look at each (by_row_scales there: 193 -> 199 us a pass at 4128 x 20480 x 3840).  Called while the MMAs run.
template <int FMT, int EPI>
ZI_DEV bool scales_mid(int row0, int lane, int n0, int half, const GemmParams& p) {
  if constexpr (FMT == NV) {
    const int col = EPI == EPI_SWIGLU ? n0 + 64 * half + 4 * lane + (lane >= 16 ? 64 : 0) : n0 + 128 * half + 4 * lane;
    auto in = [](float s) { return fabsf(s) >= 0x1p-60f && fabsf(s) <= 0x1p60f; };
    bool mid = in(__ldg(p.ars + min(row0 + lane, p.M - 1)));
    if (EPI != EPI_BF16 || col < p.N) {  // N is a multiple of 8
      const float4 w = __ldg(reinterpret_cast<const float4*>(p.brs + col));
      mid = mid && in(w.x) && in(w.y) && in(w.z) && in(w.w);
    }
    return __all_sync(0xffffffffu, mid);
  }
  return true;
}

// The epilogue of a warp's 32 rows x 128 accumulator columns, a row per lane in registers: `half` 0 or 1 of the
// 256-wide tile at column n0 (EPI_SWIGLU: v[0..63] gate columns n0 + 64 half, v[64..127] their up columns 128
// further).  The fused forms are those of gemm_epilogue: EPI_QKV one head, EPI_SWIGLU 64 outputs.  Results go
// through `stage` (the warp's 4 KB of smem), 64 columns at a time, so that 8 lanes store a row's 128 bytes: a lane
// storing its own row touches 32 lines with every instruction, and the epilogue then outlasts the next tile's MMAs
// (4128 x 20480 x 3840 NVFP4: 170 us, and 204 with a slightly longer epilogue, against 160 this way).
// MID: scales_mid of the warp.
template <int FMT, int EPI, bool MID>
ZI_DEV void wide_epilogue(uint32_t* v, int row0, int lane, int n0, int half, uint8_t* stage, const GemmParams& p,
                          const EpiParams& ep) {
  static_assert(EPI == EPI_BF16 || EPI == EPI_QKV || EPI == EPI_SWIGLU, "epilogues of the 4-bit product");
  const int nb = n0 + half * 128, m = min(row0 + lane, p.M - 1);
  const float ra = FMT == NV ? __ldg(p.ars + m) : 1.f;
  auto f = [&](int i) { return __uint_as_float(v[i]); };
  // 8 columns by their row scales
  auto scale8 = [&](int c) {
    if constexpr (FMT == NV) {
      const int col = EPI == EPI_SWIGLU ? n0 + 64 * half + 8 * c + (c >= 8 ? 64 : 0) : nb + 8 * c;
      if (EPI == EPI_BF16 && col >= p.N) return;  // N is a multiple of 8
      const float4* bs = reinterpret_cast<const float4*>(p.brs + col);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 w = __ldg(bs + h);
        uint32_t* x = v + 8 * c + 4 * h;
        auto scaled = [&](uint32_t y, float rb) {
          return __float_as_uint(MID ? __uint_as_float(y) * (ra * rb) : by_row_scales(__uint_as_float(y), ra, rb));
        };
        x[0] = scaled(x[0], w.x);
        x[1] = scaled(x[1], w.y);
        x[2] = scaled(x[2], w.z);
        x[3] = scaled(x[3], w.w);
      }
    }
  };
  auto put = [&](int c, const float* y) {  // 8 results of this lane's row, the c-th of the 64-column piece
    *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
  };
  auto flush = [&](int col, int cols) {  // the piece to global memory, at column `col` of an output `cols` wide
    __syncwarp();
    const int x = lane & 7;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int r = 4 * e + (lane >> 3);
      const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 128 + ((x ^ (r & 7)) << 4));
      if (row0 + r < p.M && col + 8 * x < cols)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(ep.out) + size_t(row0 + r) * ep.ldo + col + 8 * x) = w;
    }
    __syncwarp();
  };
  if constexpr (EPI == EPI_SWIGLU) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      scale8(c);
      scale8(c + 8);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = f(8 * c + i) / (1.0f + __expf(-f(8 * c + i))) * f(64 + 8 * c + i);
      put(c, y);
    }
    flush(n0 / 2 + 64 * half, ep.ldo);
  }
  if constexpr (EPI == EPI_QKV) {
    const int region = n0 / ep.dim;  // 0 = q, 1 = k, 2 = v
#pragma unroll
    for (int c = 0; c < 16; ++c) scale8(c);
    if (region < 2) {
      const uint16_t* g = region == 0 ? ep.g_q : ep.g_k;
      const float2* rp = ep.rope + ep.map.tab(m + ep.row_off);  // pair j at rp[j * rope_n]
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 128; ++i) ss = fmaf(f(i), f(i), ss);
      const float r = rsqrtf(ss * (1.0f / 128.0f) + ep.eps);
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        const uint32_t gp = __ldg(reinterpret_cast<const uint32_t*>(g) + i);  // gains of dims 2i, 2i + 1
        const float a = f(2 * i) * r * __uint_as_float(gp << 16), b = f(2 * i + 1) * r * __uint_as_float(gp & 0xFFFF0000u);
        const float2 cs = __ldg(rp + size_t(i) * ep.rope_n);
        v[2 * i] = __float_as_uint(a * cs.x - b * cs.y);
        v[2 * i + 1] = __float_as_uint(a * cs.y + b * cs.x);
      }
    }
  }
  if constexpr (EPI != EPI_SWIGLU) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (EPI == EPI_BF16) scale8(8 * h + c);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = f(64 * h + 8 * c + i);
        put(c, y);
      }
      flush(nb + 64 * h, EPI == EPI_BF16 ? p.N : ep.ldo);
    }
  }
}

template <int FMT, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    gemm_wide_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB, GemmParams p,
                     EpiParams ep, TailSched sched) {
  using L = WideSmem<FMT>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);  // CTA 0: both CTAs' operands loaded
  uint64_t* empty = full + kStages;     // each CTA: its stage consumed by the pair's MMAs
  uint64_t* sc_full = empty + kStages;  // each CTA: its scales loaded
  uint64_t* sc_tmem = sc_full + kStages;  // CTA 0: both CTAs' scales in TMEM
  uint64_t* tfull = sc_tmem + kStages;  // each CTA: accumulator complete
  uint64_t* tempty = tfull + 1;         // CTA 0: both CTAs' epilogues hold the accumulator
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int unit = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sc_full[s], 1);
      mbar_init(&sc_tmem[s], 8);  // one arrival per scale warp of each CTA
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 16);  // one arrival per epilogue warp of each CTA
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmSA);
    prefetch_tmap(&tmSB);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers initialised and TMEM allocated before any remote access
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool err = device_error_set();  // an earlier kernel timed out: skip the work, still meet at the end
  const int num_m = (p.M + 255) / 256;
  WorkItem wi;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideRegsLow));
    if (warp == 0 && lane == 0 && !err) {
      uint32_t it = 0;
      bool ok = true;
      WorkWalker walk(sched, unit);
      while (ok && walk.next(wi)) {
        int m0, n0;
        tile_origin<256, 256>(sched, num_m, wi.tile, m0, n0);
        for (int kb = 0; kb < sched.kb; ++kb, ++it) {
          const uint32_t s = it % kStages, r = it / kStages;
          if (!mbar_wait(&empty[s], (r & 1u) ^ 1u, abort_flag, ZI_DEVERR_TIMEOUT_PRODUCER)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * L::kStage;
          uint8_t* sc = st + L::kA + L::kB;
          mbar_arrive_expect_tx(&sc_full[s], 3u * L::kSc);
          load_3d(sc, &tmSA, &sc_full[s], 0, kb * kStageTiles<FMT>, m0 / 128 + int(rank));
          load_3d(sc + L::kSc, &tmSB, &sc_full[s], 0, kb * kStageTiles<FMT>, n0 / 128);
          load_3d(sc + 2 * L::kSc, &tmSB, &sc_full[s], 0, kb * kStageTiles<FMT>, n0 / 128 + 1);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * (L::kA + L::kB));
          tma_load_2d_pair(st, &tmA, &full[s], kb * 128, m0 + 128 * int(rank));
          tma_load_2d_pair(st + L::kA, &tmB, &full[s], kb * 128, n0 + 128 * int(rank));
        }
      }
    } else if (warp == 1 && lane == 0 && rank == 0 && !err) {
      uint32_t it = 0;
      int local = 0;
      bool ok = true;
      WorkWalker walk(sched, unit);
      while (ok && walk.next(wi)) {
        if (!mbar_wait(tempty, (uint32_t(local) & 1u) ^ 1u, abort_flag, ZI_DEVERR_TIMEOUT_MMA)) {
          ok = false;
          break;
        }
        ++local;
        tc_fence_after();
        for (int kb = 0; kb < sched.kb; ++kb, ++it) {
          const uint32_t s = it % kStages, r = it / kStages;
          if (!mbar_wait(&full[s], r & 1u, abort_flag, ZI_DEVERR_TIMEOUT_MMA) ||
              !mbar_wait(&sc_tmem[s], r & 1u, abort_flag, ZI_DEVERR_TIMEOUT_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + s * L::kStage), b_addr = a_addr + L::kA;
          const uint32_t tsa = tmem + L::kColScale + s * L::kScaleCols, tsb = tsa + 4 * kStageTiles<FMT>;
          // columns past K are zero codes under zero scales: whole steps of 64 past it are left out
          const int ksteps = min(4, (p.K - kb * kStageK + 63) / 64);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k < ksteps) {
              const int t = FMT == MX ? k >> 1 : k;
              mma2<FMT>(tmem, smem_desc_sw128(a_addr + k * 32, 16), smem_desc_sw128(b_addr + k * 32, 16),
                        idesc<FMT>(256, 256, FMT == MX ? k & 1 : 0), tsa + 4 * t, tsb + 8 * t,
                        (kb | k) != 0 ? 1u : 0u);
            }
          }
          tc_commit_pair(&empty[s]);
        }
        if (ok) tc_commit_pair(tfull);
      }
      if (!ok) {
        tc_commit_pair_local(drain);
        volatile int never = 0;
        mbar_wait(drain, 0, &never, ZI_DEVERR_TIMEOUT_DRAIN);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideRegsScale));
    // Scale tiles of a stage to this warp's lane quarter: lane l of a tile's 4 columns holds rows l, 32 + l, 64 + l
    // and 96 + l, in every quarter.  The TMEM buffer of a stage is free whenever its smem is.
    const uint32_t quarter = uint32_t((warp & 3) * 32) << 16;
    uint32_t it = 0;
    bool ok = !err;
    WorkWalker walk(sched, unit);
    while (ok && walk.next(wi)) {
      for (int kb = 0; kb < sched.kb; ++kb, ++it) {
        const uint32_t s = it % kStages, r = it / kStages;
        if (!mbar_wait_warp(&sc_full[s], r & 1u, abort_flag, ZI_DEVERR_TIMEOUT_EPILOGUE)) {
          ok = false;
          break;
        }
        const uint4* src = reinterpret_cast<const uint4*>(smem + s * L::kStage + L::kA + L::kB) + lane;
        const uint32_t dst = tmem + quarter + L::kColScale + s * L::kScaleCols;
        uint4 w[3 * kStageTiles<FMT>];
#pragma unroll
        for (int t = 0; t < 3 * kStageTiles<FMT>; ++t) w[t] = src[t * 32];
#pragma unroll
        for (int t = 0; t < kStageTiles<FMT>; ++t) {
          tmem_st4(dst + 4 * t, w[t]);
          tmem_st4(dst + 4 * kStageTiles<FMT> + 8 * t, w[kStageTiles<FMT> + t]);
          tmem_st4(dst + 4 * kStageTiles<FMT> + 8 * t + 4, w[2 * kStageTiles<FMT> + t]);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_leader(&sc_tmem[s]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWideRegsEpi));
    const int q = warp & 3, half = (warp - 8) >> 2;
    int local = 0;
    WorkWalker walk(sched, unit);
    while (!err && walk.next(wi)) {
      int m0, n0;
      tile_origin<256, 256>(sched, num_m, wi.tile, m0, n0);
      const int row0 = m0 + 128 * int(rank) + q * 32;
      const bool mid = row0 >= p.M || scales_mid<FMT, EPI>(row0, lane, n0, half, p);
      if (!mbar_wait_warp(tfull, uint32_t(local) & 1u, abort_flag, ZI_DEVERR_TIMEOUT_EPILOGUE)) break;
      ++local;
      tc_fence_after();
      uint32_t v[128];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld32(tmem + (uint32_t(q * 32) << 16) +
                      (EPI == EPI_SWIGLU ? half * 64 + c * 32 + (c >= 2 ? 64 : 0) : half * 128 + c * 32),
                  &v[c * 32]);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) reg_fence32(&v[c * 32]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(tempty);
      uint8_t* stage = smem + L::kOut + (warp - 8) * 4096;
      if (row0 >= p.M) continue;
      if (FMT == MX || mid)
        wide_epilogue<FMT, EPI, true>(v, row0, lane, n0, half, stage, p, ep);
      else
        wide_epilogue<FMT, EPI, false>(v, row0, lane, n0, half, stage, p, ep);
    }
  }

  if (*abort_flag) {  // an aborted pipeline: let copies already issued land before the pair leaves
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA frees TMEM or exits while the pair's MMAs or copies may use it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

}  // namespace fp4
}  // namespace zi
