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
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
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
  __device__ __forceinline__ void store(__half* p) const { *reinterpret_cast<uint4*>(p) = a; }
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
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
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
// 16 elements, in accesses of 32 bytes where `wide` (the address is so aligned):
// a warp's 16-byte accesses 32 bytes apart would touch every sector twice.
__device__ __forceinline__ void ld_global32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ void st_global32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void load16(Raw8<T>* r, const T* x, int wide) {
  if (wide) {
    if constexpr (sizeof(T) == 2) {
      ld_global32(x, r[0].a, r[1].a);
    } else {
      ld_global32(x, reinterpret_cast<uint4&>(r[0].a), reinterpret_cast<uint4&>(r[0].b));
      ld_global32(x + 8, reinterpret_cast<uint4&>(r[1].a), reinterpret_cast<uint4&>(r[1].b));
    }
  } else {
    r[0].load(x);
    r[1].load(x + 8);
  }
}
__device__ __forceinline__ uint4 pack8(const __nv_bfloat16*, const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack8(const __half*, const float* v) {
  return make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
}
template <typename T>
__device__ __forceinline__ void store16(T* y, const float* v, int wide) {
  if (!wide) {
    store8(y, v);
    store8(y + 8, v + 8);
  } else if constexpr (sizeof(T) == 2) {
    st_global32(y, pack8(y, v), pack8(y, v + 8));
  } else {
    const uint4* u = reinterpret_cast<const uint4*>(v);
    st_global32(y, u[0], u[1]);
    st_global32(y + 8, u[2], u[3]);
  }
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

// ---------------------------------------------------------------- arithmetic
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if one of them is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Both factors of each of four pairs of v times m.
__device__ __forceinline__ void scale8(const float* v, float m, float* r) {
  const uint64_t mm = f2_pack(m, m);
#pragma unroll
  for (int i = 0; i < 8; i += 2) f2_unpack(f2_mul(f2_pack(v[i], v[i + 1]), mm), r[i], r[i + 1]);
}

// ---------------------------------------------------------------- conversions
// Four floats to e4m3 / eight to e2m1 (nearest, ties to even, at most the
// largest finite value); element 0 in the lowest bits.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}
__device__ __forceinline__ uint32_t e2m1x8(const float* v, float m) {  // of v m
  float f[8];
  scale8(v, m, f);
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
__device__ __forceinline__ uint2 e4m3x8(const float* v, float m) {  // of v m
  float f[8];
  scale8(v, m, f);
  return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
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

// The border between the e2m1 codes c and c + 1, c = 0 .. 6 (half the sum of
// their values: 1, 3, 5, 7, 10, 14, 20 quarters).
__device__ __forceinline__ float e2m1_border(uint32_t c) {
  return 0.25f * static_cast<float>(static_cast<uint32_t>(0x140e0a07050301ull >> (8 * c)) & 0xffu);
}

// Eight elements of an nvfp4 block with scale value s (inv ~ 1 / (s g) within
// 3 2^-24; the product with v and that with 1 -+ 2^-21 add 2^-24 each):
// nearest e2m1 of v / (s g), exactly, by the same two conversions; where they differ, the element's border's product border * s (7 bits) decides
// by the sign of one fma, and a tie goes to the even code. (Ties are common
// where g is a short number: bf16 inputs have 8 bits. So the loop takes only
// the elements that differ; a pass over all eight cost 30 us at 51200 x 2304.)
__device__ __forceinline__ uint32_t nvfp4_elements(const float* v, float s, float g, float inv) {
  uint32_t lo = e2m1x8(v, inv * kBelow);
  const uint32_t x = lo ^ e2m1x8(v, inv * kAbove);
  for (uint32_t m = (x | x >> 1 | x >> 2) & 0x11111111u; m != 0; m &= m - 1) {
    const int at = __ffs(m) - 1;  // 4 i
    const bool b0 = at & 4, b1 = at & 8, b2 = at & 16;
    const float v01 = b0 ? v[1] : v[0], v23 = b0 ? v[3] : v[2], v45 = b0 ? v[5] : v[4], v67 = b0 ? v[7] : v[6];
    const float vi = b2 ? (b1 ? v67 : v45) : (b1 ? v23 : v01);
    const uint32_t c = (lo >> at) & 7u;
    const float d = fmaf(-(e2m1_border(c) * s), g, fabsf(vi));
    if (d > 0.f || (d == 0.f && (c & 1u))) lo += 1u << at;
  }
  return lo;
}

// Largest magnitude of 16 loaded elements as the bits of an fp32 number
// (16-bit magnitudes order as their bits do, infinities and NaN on top).
__device__ __forceinline__ uint32_t amax16_bits(const uint4& a, const uint4& b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  return max(m & 0xffffu, m >> 16);
}
__device__ __forceinline__ uint32_t amax16(const Raw8<__nv_bfloat16>& a, const Raw8<__nv_bfloat16>& b, const float*) {
  return amax16_bits(a.a, b.a) << 16;
}
__device__ __forceinline__ uint32_t amax16(const Raw8<__half>& a, const Raw8<__half>& b, const float*) {
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(amax16_bits(a.a, b.a)))));
}
__device__ __forceinline__ uint32_t amax16(const Raw8<float>&, const Raw8<float>&, const float* v) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) m = max_nan(m, fabsf(v[e]));
  return __float_as_uint(m);
}

// ---------------------------------------------------------------- rows in groups of 128
// Quotient by a divisor fixed at launch, for u < 2^31: with l = ceil(log2 d) and
// m = ceil(2^(31 + l) / d), u / d = (u m) >> (31 + l); d >= 2.
struct FastDiv {
  uint32_t m, s;
  __device__ __forceinline__ uint32_t div(uint32_t u) const { return __umulhi(u, m) >> s; }
};

// A thread of both kernels below takes one unit of 16 consecutive elements of
// four rows, 32 apart: their scales share 16 bytes of a tile, so that scales
// move in whole 16-byte words, and four loads are in flight. Position t of the
// grid is unit t % upr of rows (t / upr) / 32 * 128 + (t / upr) % 32 + 32 i.
constexpr int kMxRows = 4;

// ---------------------------------------------------------------- quantisation of rows
struct MxQuantParams {
  const void* X;      // [B, N, D]
  const int32_t* S;   // [B, R] rows, or null
  uint8_t* data;      // [B * R, D or D / 2]
  uint8_t* scales;    // tiles
  float g, inv6g;
  int N, R, D;
  int ct;             // scale tiles along a row
  int upr;            // 16-element units of a row, up to whole scale tiles
  int rows, row0;     // B * R; the launch's first row
  uint32_t threads;   // positions of the launch
  int wide;           // X is 32-byte aligned
  FastDiv by_upr, by_R;
};

// Bound by memory: x is read once, elements and scales are written once.
// Measured (bf16, 51200 x 2304): mxfp8 59 us, mxfp4 52 us, nvfp4 61 us (6.0,
// 5.7, 4.9 TB/s). A thread for one unit of one row, with 64-bit divisions for
// its place, took 72, 70 and 82 us.
template <typename T, int kFmt>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const MxQuantParams p) {
  pdl_launch_dependents();  // a dependent layer may set up meanwhile
  const uint32_t t = blockIdx.x * 256 + threadIdx.x;
  // the grid's last positions past the end repeat the last one, without stores
  const bool live = t < p.threads;
  const uint32_t tt = live ? t : p.threads - 1, rr = p.by_upr.div(tt);
  const int unit = static_cast<int>(tt - rr * p.upr);
  const int r0 = p.row0 + static_cast<int>((rr >> 5) * 128 + (rr & 31));
  const bool in = unit * 16 < p.D;
  Raw8<T> raw[kMxRows][2];
#pragma unroll
  for (int i = 0; i < kMxRows; ++i) {
    const int row = r0 + 32 * i;
    raw[i][0].zero();
    raw[i][1].zero();
    if (in && row < p.rows) {
      long long src = row;
      if (p.S != nullptr) {
        int idx = __ldg(p.S + row);
        if (idx < 0 || idx >= p.N) {
          if (unit == 0 && live) raise_status(1 << 5);
          idx = 0;
        }
        src = (p.R == 1 ? row : static_cast<long long>(p.by_R.div(row))) * p.N + idx;
      }
      const T* x = static_cast<const T*>(p.X) + src * p.D + unit * 16;
      load16(raw[i], x, p.wide);
    }
  }
  constexpr int kLanes = kFmt == kNvFp4 ? 4 : 8;  // lanes whose scales make a word: 4 scales of one row
  uint32_t words[kMxRows];
#pragma unroll
  for (int i = 0; i < kMxRows; ++i) {
    const int row = r0 + 32 * i;
    float v[16];
    raw[i][0].get(v);
    raw[i][1].get(v + 8);
    uint32_t amax = amax16(raw[i][0], raw[i][1], v), byte, out[4];
    if constexpr (kFmt == kNvFp4) {
      byte = nvfp4_scale(amax, p.g, p.inv6g);
      const float s = e4m3_value(byte);
      const float inv = byte == 0 || byte == 0x7fu ? 0.f : rcp_approx(s * p.g);
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
        const uint2 lo = e4m3x8(v, inv), hi = e4m3x8(v + 8, inv);
        out[0] = lo.x;
        out[1] = lo.y;
        out[2] = hi.x;
        out[3] = hi.y;
      }
    }
    // this row's word of scales; those past the row or the matrix are zero
    const int at = kFmt == kNvFp4 ? threadIdx.x & 3 : (threadIdx.x >> 1) & 3;
    uint32_t word = in && row < p.rows ? byte << (8 * at) : 0u;
    if constexpr (kFmt == kNvFp4) word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    if constexpr (kFmt != kNvFp4) word |= __shfl_xor_sync(0xffffffffu, word, 4);
    words[i] = word;
    if (live && in && row < p.rows) {
      if constexpr (kFmt == kMxFp8)
        *reinterpret_cast<uint4*>(p.data + static_cast<size_t>(row) * p.D + unit * 16) =
            make_uint4(out[0], out[1], out[2], out[3]);
      else
        *reinterpret_cast<uint2*>(p.data + static_cast<size_t>(row) * (p.D / 2) + unit * 8) = make_uint2(out[0], out[1]);
    }
  }
  if (live && (threadIdx.x & (kLanes - 1)) == 0)
    *reinterpret_cast<uint4*>(p.scales + mx_scale_at(r0, unit / (kLanes / 4), p.ct)) =
        make_uint4(words[0], words[1], words[2], words[3]);
}

// ---------------------------------------------------------------- decoding
struct MxDecodeParams {
  const uint8_t* data;
  const uint8_t* scales;
  void* Y;  // [rows, D]
  float g;
  int D, ct, upr, rows, row0;  // upr = D / 16
  int wide;                    // Y is 32-byte aligned
  uint32_t threads;
  FastDiv by_upr;
};

// value = element * scale * g: the product of element and scale is exact in
// fp32, the factor g rounds once, the conversion to the output type once.
// Bound by memory. Measured (to bf16, 51200 x 2304): mxfp8 59 us, mxfp4 and
// nvfp4 51 us (5.8 - 6.0 TB/s); with stores of 16 bytes, two to a sector, 68 and
// 70 us.
template <typename T, int kFmt>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const MxDecodeParams p) {
  const uint32_t t = blockIdx.x * 256 + threadIdx.x;
  if (t >= p.threads) return;
  const uint32_t rr = p.by_upr.div(t);
  const int unit = static_cast<int>(t - rr * p.upr);
  const int r0 = p.row0 + static_cast<int>((rr >> 5) * 128 + (rr & 31));
  const int j = kFmt == kNvFp4 ? unit : unit >> 1;
  const uint4 sw = __ldg(reinterpret_cast<const uint4*>(p.scales + mx_scale_at(r0, j & ~3, p.ct)));
  const uint32_t words[4] = {sw.x, sw.y, sw.z, sw.w};
  uint4 raw[kMxRows];
#pragma unroll
  for (int i = 0; i < kMxRows; ++i) {
    const int row = r0 + 32 * i;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (row < p.rows) {
      if constexpr (kFmt == kMxFp8) {
        raw[i] = __ldg(reinterpret_cast<const uint4*>(p.data + static_cast<size_t>(row) * p.D + unit * 16));
      } else {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(p.data + static_cast<size_t>(row) * (p.D / 2) + unit * 8));
        raw[i].x = a.x;
        raw[i].y = a.y;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kMxRows; ++i) {
    const int row = r0 + 32 * i;
    if (row >= p.rows) break;
    const uint32_t byte = (words[i] >> (8 * (j & 3))) & 0xffu;
    const float s = kFmt == kNvFp4 ? e4m3_value(byte) : e8m0_value(byte);
    float v[16];
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // two elements
      uint32_t h2;
      if constexpr (kFmt == kMxFp8) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)))));
      } else {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
            : "=r"(h2)
            : "r"(w[e / 4] >> (8 * (e & 3))));
      }
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      v[2 * e] = f.x * s;
      v[2 * e + 1] = f.y * s;
      if constexpr (kFmt == kNvFp4) {
        v[2 * e] *= p.g;
        v[2 * e + 1] *= p.g;
      }
    }
    T* y = static_cast<T*>(p.Y) + static_cast<size_t>(row) * p.D + unit * 16;
    store16(y, v, p.wide);
  }
}

}  // namespace safe
