// norm.cuh - root-mean-square norm of rows, with the residual's addition and an
// output in 8 bits.
//
// The norms between the branches of the block B (Eq. (18)) and of its
// row-selective form B^S (Eq. (15)):
//     h = x + res,   y = h / sqrt(mean(h^2) + eps) * w
// h is the residual stream after the branch, y the next branch's input.
// With the rows S of Eq. (13), row r of the output belongs to token S[b, r].
// The sum h is held in fp32 for the norm; only its copy in the stream is
// rounded to the stream's type. The 8-bit output quantises the fp32 y in
// blocks of 32 (mx_quant.cuh) without a rounding in between.
#pragma once

#include "mx_quant.cuh"

namespace safe {

struct NormParams {
  const void* x;     // [B, R, D], or [B, N, D] with x_full
  const void* res;   // [B, N, D] or null
  const int32_t* S;  // [B, R] or null
  const float* w;    // [D] or null
  void* h;           // [B, R, D], or [B, N, D] with h_full; null: not written
  void* y;           // [B, R, D] or null
  uint8_t* q;        // [B * R, D] e4m3 or null
  uint8_t* q_scales;
  float eps;
  int N, R, D, x_full, h_full, ct;
  long long rows, rows_pad;  // B * R; with q up to a multiple of 128
};

// Rows of a tensor for output row `row`; false: a bad index (flagged), the
// row's outputs are zeros and the stream's row is left as it was. In place
// (h_full with S) two equal rows would race, so there S has to ascend.
__device__ __forceinline__ bool norm_rows(const NormParams& p, long long row, bool flag, long long& xr, long long& rr,
                                          long long& hr) {
  xr = rr = hr = row;
  if (p.S == nullptr) return true;
  const long long b = row / p.R;
  const int r = static_cast<int>(row - b * p.R);
  const int idx = __ldg(p.S + row);
  bool ok = idx >= 0 && idx < p.N;
  if (p.h_full && r > 0 && __ldg(p.S + row - 1) >= idx) ok = false;
  if (!ok && flag) raise_status(1 << 5);
  const long long full = b * p.N + idx;
  if (p.x_full) xr = full;
  rr = full;
  if (p.h_full) hr = full;
  return ok;
}

// Sum over the TPR threads of a row (every thread gets it).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += part[i];
  }
  return v;
}

// TPR threads take a row, each NV units of VEC consecutive elements, and keep
// it in registers between the sum and the output: one read of x and res.
// VEC = 8 where rows and tensors are 16-byte aligned, else 1.
template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) rms_norm_kernel(const NormParams p) {
  constexpr int kRowsCta = TPR < 128 ? 128 / TPR : 1;
  __shared__ float part[TPR / 32];
  const int t = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * kRowsCta + threadIdx.x / TPR;
  if (row >= p.rows_pad) return;  // whole rows leave: whole warps, or the CTA
  const int units = p.D / VEC;
  if (row >= p.rows) {  // fills the last scale tile up
    for (int j = 4 * t; j < 4 * p.ct; j += 4 * TPR)
      *reinterpret_cast<uint32_t*>(p.q_scales + mx_scale_at(row, j, p.ct)) = 0u;
    return;
  }
  long long xr, rr, hr;
  const bool ok = norm_rows(p, row, t == 0, xr, rr, hr);
  const T* x = static_cast<const T*>(p.x) + (ok ? xr : 0) * p.D;
  const T* res = p.res != nullptr ? static_cast<const T*>(p.res) + (ok ? rr : 0) * p.D : nullptr;
  T* h = p.h != nullptr ? static_cast<T*>(p.h) + (ok ? hr : p.h_full ? 0 : row) * p.D : nullptr;
  const bool h_write = p.h != nullptr && (ok || !p.h_full);

  float v[NV * VEC];
  if constexpr (VEC == 8) {
    Raw8<T> a[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = i * TPR + t;
      a[i].zero();
      if (ok && u < units) a[i].load(x + u * 8);
    }
    if (res != nullptr) {
      Raw8<T> b[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int u = i * TPR + t;
        b[i].zero();
        if (ok && u < units) b[i].load(res + u * 8);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8];
        a[i].get(v + 8 * i);
        b[i].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * i + e] += f[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) a[i].get(v + 8 * i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = i * TPR + t;
      v[i] = ok && u < units ? to_float(x[u]) : 0.f;
    }
    if (res != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int u = i * TPR + t;
        if (ok && u < units) v[i] += to_float(res[u]);
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV * VEC; ++i) ss = fmaf(v[i], v[i], ss);
  ss = row_sum<TPR>(ss, part);
  const float rstd = ok ? 1.f / sqrtf(ss / static_cast<float>(p.D) + p.eps) : 0.f;

  T* y = p.y != nullptr ? static_cast<T*>(p.y) + row * p.D : nullptr;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int u = i * TPR + t;
    const bool in = u < units;
    if constexpr (VEC == 8) {
      if (in && h_write) store8(h + u * 8, v + 8 * i);
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = v[8 * i + e] * rstd;
      if (in && p.w != nullptr) {
        const float4 w0 = __ldg(reinterpret_cast<const float4*>(p.w) + 2 * u);
        const float4 w1 = __ldg(reinterpret_cast<const float4*>(p.w) + 2 * u + 1);
        f[0] *= w0.x; f[1] *= w0.y; f[2] *= w0.z; f[3] *= w0.w;
        f[4] *= w1.x; f[5] *= w1.y; f[6] *= w1.z; f[7] *= w1.w;
      }
      if (!ok) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
      }
      if (in && y != nullptr) store8(y + u * 8, f);
      if (p.q != nullptr) {
        // blocks of 32: four threads; a word of scales: sixteen (D is a
        // multiple of 32, so a block is inside the row or past its end)
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(f[e]) & 0x7fffffffu);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float inv;
        uint32_t word = e8m0_scale<8>(amax, inv);
        if (!in) word = 0;
        word <<= 8 * ((t >> 2) & 3);
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if (in) {
          *reinterpret_cast<uint2*>(p.q + row * p.D + u * 8) =
              make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                         e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
          if ((t & 15) == 0) *reinterpret_cast<uint32_t*>(p.q_scales + mx_scale_at(row, u >> 2, p.ct)) = word;
        }
      }
    } else {
      if (in) {
        if (h_write) h[u] = from_float<T>(v[i]);
        const float f = ok ? (p.w != nullptr ? v[i] * rstd * __ldg(p.w + u) : v[i] * rstd) : 0.f;
        if (y != nullptr) y[u] = from_float<T>(f);
      }
    }
  }
}

// Rows too long for the registers: 512 threads read the row twice. In place
// each element is read and written by one thread, in this order.
template <typename T>
__global__ void __launch_bounds__(512) rms_norm_long_kernel(const NormParams p) {
  __shared__ float part[16];
  const long long row = blockIdx.x;
  long long xr, rr, hr;
  const bool ok = norm_rows(p, row, threadIdx.x == 0, xr, rr, hr);
  const T* x = static_cast<const T*>(p.x) + (ok ? xr : 0) * p.D;
  const T* res = p.res != nullptr ? static_cast<const T*>(p.res) + (ok ? rr : 0) * p.D : nullptr;
  T* h = p.h != nullptr ? static_cast<T*>(p.h) + (ok ? hr : p.h_full ? 0 : row) * p.D : nullptr;
  const bool h_write = p.h != nullptr && (ok || !p.h_full);
  T* y = p.y != nullptr ? static_cast<T*>(p.y) + row * p.D : nullptr;
  float ss = 0.f;
  if (ok)
    for (int u = threadIdx.x; u < p.D; u += 512) {
      float v = to_float(x[u]);
      if (res != nullptr) v += to_float(res[u]);
      ss = fmaf(v, v, ss);
    }
  ss = row_sum<512>(ss, part);
  const float rstd = ok ? 1.f / sqrtf(ss / static_cast<float>(p.D) + p.eps) : 0.f;
  for (int u = threadIdx.x; u < p.D; u += 512) {
    float v = 0.f;
    if (ok) {
      v = to_float(x[u]);
      if (res != nullptr) v += to_float(res[u]);
    }
    if (h_write) h[u] = from_float<T>(v);
    if (y != nullptr) y[u] = from_float<T>(ok ? (p.w != nullptr ? v * rstd * __ldg(p.w + u) : v * rstd) : 0.f);
  }
}

}  // namespace safe
