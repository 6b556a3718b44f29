// mx_quant.cuh - microscaled rows: element and scale formats, quantisation, decoding.
//
// A microscaled matrix [rows, D] holds one scale for each block of
// consecutive elements of a row:
//   SAFE_MXFP8  e4m3 elements, blocks of 32, scale 2^e (e8m0)
//   SAFE_MXFP4  e2m1 elements, blocks of 32, scale 2^e (e8m0)
//   SAFE_NVFP4  e2m1 elements, blocks of 16, scale e4m3, and one fp32 factor g
//               for the whole tensor
// value = element * scale (* g). Elements are row-major (two e2m1 to a byte,
// the even element in the low half). Scale bytes lie in the order in which
// the tensor core takes them: tiles of 128 rows x 4 scales of 512 bytes, the
// tiles of 128 rows one after another along the row; within a tile row i and
// scale j at byte (i % 32) 16 + (i / 32) 4 + j. Rows and scales that only
// fill a tile up are zero.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "sm100.cuh"

namespace safe {

enum : int { kMxFp8 = 0, kMxFp4 = 1, kNvFp4 = 2 };

// Byte of scale j of row `row`; ct = tiles along a row.
__device__ __forceinline__ size_t mx_scale_at(size_t row, int j, int ct) {
  return ((row >> 7) * ct + (j >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (j & 3);
}

// ---------------------------------------------------------------- loads and stores of 8 elements
template <typename T>
struct Raw8;  // 8 elements of T as loaded (16 bytes for the 16-bit types, 32 for fp32)
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<__half> {
  uint4 a;
  __device__ __forceinline__ void load(const __half* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(__half* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                                            pack_f16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }

// ---------------------------------------------------------------- conversions
// Four floats to e4m3 / eight to e2m1 (nearest, ties to even, at most the
// largest finite value); element 0 in the lowest bits.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}
__device__ __forceinline__ uint32_t e2m1x8(const float* v, float m) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0] * m), "f"(v[1] * m), "f"(v[2] * m), "f"(v[3] * m), "f"(v[4] * m), "f"(v[5] * m), "f"(v[6] * m),
        "f"(v[7] * m));
  return r;
}
// The value of an e4m3 byte (0x7f and 0xff are NaN).
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(byte & 0xffu)));
  return __low2float(*reinterpret_cast<const __half2*>(&h2));
}
__device__ __forceinline__ uint32_t e4m3_byte(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
// 2^(byte - 127), the value of an e8m0 byte (0 is the subnormal 2^-127, 255 is NaN).
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7fffffffu : byte << 23);
}

// Power-of-two scale of a block whose largest magnitude has the bits `amax`
// (sign cleared): e = floor(log2 amax) - kTop, kTop the exponent of the
// element type's largest value (8 for e4m3, 2 for e2m1), within e8m0's range;
// magnitudes above the largest element value saturate. A block of zeros gets
// 2^-127, one with an infinity or a NaN the NaN byte. Every step is exact, and
// so is x * `inverse` (a power of two).
template <int kTop>
__device__ __forceinline__ uint32_t e8m0_scale(uint32_t amax, float& inverse) {
  const int e = static_cast<int>(amax >> 23);
  if (e == 255) {
    inverse = 0.f;
    return 255u;
  }
  const int byte = e > kTop ? e - kTop : 0;
  inverse = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
  return static_cast<uint32_t>(byte);
}

// The e4m3 scale of an nvfp4 block: nearest e4m3 of amax / (6 g), exactly.
// amax * inv6g is within 2^-22 of the quotient; where the conversions of that
// value times 1 -+ 2^-21 differ, a rounding border lies between them, and
// the sign of amax - border * 6 g decides: border * 6 has 8 bits at most, so
// one fma gives that sign without error.
constexpr float kBelow = 1.f - 4.76837158203125e-07f, kAbove = 1.f + 4.76837158203125e-07f;  // 1 -+ 2^-21
__device__ __forceinline__ uint32_t nvfp4_scale(uint32_t amax_bits, float g, float inv6g) {
  if (amax_bits >= 0x7f800000u) return 0x7fu;
  const float amax = __uint_as_float(amax_bits), r = amax * inv6g;
  const uint32_t lo = e4m3_byte(r * kBelow), hi = e4m3_byte(r * kAbove);
  if (lo == hi) return lo;
  const float border6 = 3.f * (e4m3_value(lo) + e4m3_value(hi));
  const float d = fmaf(-border6, g, amax);
  return d > 0.f ? hi : d < 0.f ? lo : (lo & 1u) ? hi : lo;
}

// The e2m1 magnitudes' borders: code c (0..6) and c + 1 meet at half the sum of
// their values, and a tie goes to the even code.
__device__ __forceinline__ float e2m1_border(uint32_t c) {
  return c < 3 ? 0.25f + 0.5f * c : c == 3 ? 1.75f : c == 4 ? 2.5f : c == 5 ? 3.5f : 5.f;
}

// Eight elements of an nvfp4 block with scale value s (inv ~ 1 / (s g) within
// 2^-22): nearest e2m1 of v / (s g), exactly, by the same two conversions;
// where they differ for some element, its border's product border * s (7
// bits) decides by the sign of one fma.
__device__ __forceinline__ uint32_t nvfp4_elements(const float* v, float s, float g, float inv) {
  uint32_t lo = e2m1x8(v, inv * kBelow);
  const uint32_t hi = e2m1x8(v, inv * kAbove);
  if (lo != hi) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = (lo >> (4 * i)) & 7u, b = (hi >> (4 * i)) & 7u;
      if (a != b) {
        const float d = fmaf(-(e2m1_border(a) * s), g, fabsf(v[i]));
        if (d > 0.f || (d == 0.f && (a & 1u))) lo += 1u << (4 * i);
      }
    }
  }
  return lo;
}

// ---------------------------------------------------------------- quantisation of rows
struct MxQuantParams {
  const void* X;      // [B, N, D]
  const int32_t* S;   // [B, R] rows, or null
  uint8_t* data;      // [B * R, D or D / 2]
  uint8_t* scales;    // tiles
  float g, inv6g;
  int B, N, R, D;
  int ct;             // scale tiles along a row
  int upr;            // 16-element units of a row, a multiple of 4 (those past D only fill the scale tiles up)
  long long rows;     // B * R
  long long rows_pad; // up to a multiple of 128
};

// Thread = one unit of 16 consecutive elements: a whole block of nvfp4, half of
// one of 32. Bound by memory: x is read once, the elements and scales are
// written once.
constexpr int kMxUnroll = 4;
template <typename T, int kFmt>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const MxQuantParams p) {
  const long long total = p.rows_pad * p.upr;
  const long long u0 = static_cast<long long>(blockIdx.x) * (256 * kMxUnroll) + threadIdx.x;
  Raw8<T> raw[kMxUnroll][2];
  long long row[kMxUnroll];
  int unit[kMxUnroll];
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    const long long u = u0 + 256 * i;
    raw[i][0].zero();
    raw[i][1].zero();
    row[i] = u < total ? u / p.upr : -1;
    unit[i] = static_cast<int>(u - row[i] * p.upr);
    if (row[i] >= 0 && row[i] < p.rows && unit[i] * 16 < p.D) {
      long long src = row[i];
      if (p.S != nullptr) {
        int idx = __ldg(p.S + row[i]);
        if (idx < 0 || idx >= p.N) {
          if (unit[i] == 0) raise_status(1 << 5);
          idx = 0;
        }
        src = (row[i] / p.R) * p.N + idx;
      }
      const T* x = static_cast<const T*>(p.X) + src * p.D + unit[i] * 16;
      raw[i][0].load(x);
      raw[i][1].load(x + 8);
    }
  }
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    // every lane takes the shuffles; lanes of four hold 64 elements of one row
    float v[16];
    raw[i][0].get(v);
    raw[i][1].get(v + 8);
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = max(amax, __float_as_uint(v[e]) & 0x7fffffffu);
    uint32_t byte, out[4];
    if constexpr (kFmt == kNvFp4) {
      byte = nvfp4_scale(amax, p.g, p.inv6g);
      const float s = e4m3_value(byte);
      const float inv = byte == 0 || byte == 0x7fu ? 0.f : __frcp_rn(s * p.g);
      out[0] = nvfp4_elements(v, s, p.g, inv);
      out[1] = nvfp4_elements(v + 8, s, p.g, inv);
    } else {
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      float inv;
      byte = e8m0_scale<kFmt == kMxFp8 ? 8 : 2>(amax, inv);
      if constexpr (kFmt == kMxFp4) {
        out[0] = e2m1x8(v, inv);
        out[1] = e2m1x8(v + 8, inv);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          out[e] = e4m3x4(v[4 * e] * inv, v[4 * e + 1] * inv, v[4 * e + 2] * inv, v[4 * e + 3] * inv);
      }
    }
    // the scale bytes of the four lanes: four of nvfp4 (one word), two of the others (half a word)
    if (unit[i] * 16 >= p.D || row[i] >= p.rows) byte = 0;
    uint32_t word = byte << (8 * (threadIdx.x & 3));
    if constexpr (kFmt != kNvFp4) word = byte << (8 * ((threadIdx.x & 3) >> 1));
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    if (row[i] < 0) continue;
    if ((threadIdx.x & 3) == 0) {
      if constexpr (kFmt == kNvFp4)
        *reinterpret_cast<uint32_t*>(p.scales + mx_scale_at(row[i], unit[i], p.ct)) = word;
      else
        *reinterpret_cast<uint16_t*>(p.scales + mx_scale_at(row[i], unit[i] >> 1, p.ct)) = static_cast<uint16_t>(word);
    }
    if (row[i] >= p.rows || unit[i] * 16 >= p.D) continue;
    if constexpr (kFmt == kMxFp8)
      *reinterpret_cast<uint4*>(p.data + row[i] * p.D + unit[i] * 16) = make_uint4(out[0], out[1], out[2], out[3]);
    else
      *reinterpret_cast<uint2*>(p.data + row[i] * (p.D / 2) + unit[i] * 8) = make_uint2(out[0], out[1]);
  }
}

// ---------------------------------------------------------------- decoding
struct MxDecodeParams {
  const uint8_t* data;
  const uint8_t* scales;
  void* Y;  // [rows, D]
  float g;
  int D, ct, upr;  // upr = D / 16
  long long units;
};

// value = element * scale * g: the product of element and scale is exact in
// fp32, the factor g rounds once, the conversion to the output type once.
template <typename T, int kFmt>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const MxDecodeParams p) {
  const long long u = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (u >= p.units) return;
  const long long row = u / p.upr;
  const int unit = static_cast<int>(u - row * p.upr);
  float v[16], s;
  if constexpr (kFmt == kNvFp4)
    s = e4m3_value(p.scales[mx_scale_at(row, unit, p.ct)]);
  else
    s = e8m0_value(p.scales[mx_scale_at(row, unit >> 1, p.ct)]);
  if constexpr (kFmt == kMxFp8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p.data + row * p.D + unit * 16);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(p.data + row * (p.D / 2) + unit * 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      // e2m1: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 by their twofold in four bits each
      const uint32_t c = ((i < 8 ? a.x : a.y) >> (4 * (i & 7))) & 15u;
      const float m = 0.5f * static_cast<float>((0xC8643210u >> (4 * (c & 7u))) & 15u);
      v[i] = c & 8u ? -m : m;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = v[i] * s * p.g;
  T* y = static_cast<T*>(p.Y) + row * p.D + unit * 16;
  store8(y, v);
  store8(y + 8, v + 8);
}

}  // namespace safe
