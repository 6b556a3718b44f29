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
  const uint8_t* mark;  // in place: a byte of row r at mark + r * mark_pitch, 1: out of order; or null
  size_t mark_pitch;
  float eps, inv_D;
  int N, R, D, x_full, h_full, ct;
  int rows, rows_pad;  // B * R; with q up to a multiple of 128
  FastDiv by_R;
};

// In place (h_full with S) two rows of one index would race for the stream's
// row, so a row counts only where its index lies above every earlier one of its
// sample: at most one row of an index does. This kernel runs ahead of the norm and
// leaves a byte for each row where the norm will write that row's y (or q), which the
// norm reads first. A CTA marks `per` rows of a sample (a multiple of 1024), after
// the largest of all the indices in front of them, so that no CTA waits for
// another: CTAs times rows reads in all, and so 128 CTAs at most (25600 rows in 25
// CTAs: 1.3 MB). Measured (bf16, two samples, D = 2304, to 8 bits, with / without the
// update in place): 6400 rows each 50 / 45 us, 1229 each 19.5 / 16.4; 64 rows of one
// sample 9.2 / 8.2.
constexpr int kNormOrderCtas = 128;
__global__ void __launch_bounds__(1024)
    norm_order_kernel(const int32_t* S, uint32_t R, uint32_t per, uint8_t* mark, size_t pitch) {
  __shared__ int before[32], own[2][32];
  pdl_launch_dependents();  // the norm may start: it waits for the marks only
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t first = blockIdx.x * per, end = R - first < per ? R : first + per;
  S += static_cast<size_t>(blockIdx.y) * R;
  mark += static_cast<size_t>(blockIdx.y) * R * pitch;
  int top = -1;  // the largest index in front of the next 1024 rows
  for (uint32_t i = threadIdx.x; i < first; i += 1024) top = max(top, S[i]);
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) before[warp] = top;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, before[lane]);
  for (uint32_t at = first, turn = 0; at < end; at += 1024, turn ^= 1) {
    const uint32_t r = at + threadIdx.x;
    const int idx = r < end ? S[r] : -1;
    int upto = idx;  // the largest of the warp's indices up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto = max(upto, v);
    }
    if (lane == 31) own[turn][warp] = upto;
    __syncthreads();
    const int other = own[turn][lane], left = __shfl_up_sync(0xffffffffu, upto, 1);
    int front = max(top, __reduce_max_sync(0xffffffffu, lane < warp ? other : -1));
    if (lane > 0) front = max(front, left);
    if (r < end) mark[r * pitch] = idx <= front;
    top = max(top, __reduce_max_sync(0xffffffffu, other));
  }
}

// Rows of a tensor for output row `row`; false: a bad index (flagged), the
// row's outputs are zeros and the stream's row is left as it was.
__device__ __forceinline__ bool norm_rows(const NormParams& p, int row, bool flag, int& xr, int& rr, int& hr) {
  xr = rr = hr = row;
  if (p.S == nullptr) return true;
  const int b = p.R == 1 ? row : static_cast<int>(p.by_R.div(row)), r = row - b * p.R;
  const int idx = __ldg(p.S + row);
  const bool ok = idx >= 0 && idx < p.N;
  if (!ok && flag) raise_status(1 << 5);
  const int full = b * p.N + idx;  // B N <= INT_MAX
  if (p.x_full) xr = full;
  rr = full;
  if (p.h_full) hr = full;
  return ok;
}

// Whether a row is in order; taken behind the loads, which need not wait for the
// marks, and ahead of everything that writes. Rows of a bad index take it too: the
// zeros of their y must not be in memory before their mark.
__device__ __forceinline__ bool norm_in_order(const NormParams& p, int row, bool flag) {
  if (p.mark == nullptr) return true;
  pdl_wait();
  const bool ok = p.mark[row * p.mark_pitch] == 0;
  if (!ok && flag) raise_status(1 << 5);
  return ok;
}

// Sum over the TPR threads of a row (every thread gets it).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = TPR < 32 ? TPR / 2 : 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += part[i];
  }
  return v;
}

// How the elements of a row are accessed:
//   kNormVec    8 at a time; rows and tensors 16-byte aligned (D a multiple of 8)
//   kNormShift  8 at a time from the aligned address at or before the row's
//               first element, for any D, where every tensor has its row at
//               the same place (no S) and begins 16-byte aligned; elements of
//               the neighbouring rows are masked, edges stored one by one
//   kNormOne    one by one
// Measured (bf16 with the residual, 51200 rows): D = 2304 143 us (6.6 TB/s),
// 2303 190 us shifted, 472 one by one.
enum : int { kNormVec, kNormShift, kNormOne };

// TPR threads take a row, each NV units of 8 elements (one in kNormOne), and keep
// it in registers between the sum and the output: one read of x and res. Bound
// by memory, and with the 8-bit output by issue. Few registers for each thread
// and many rows at once keep more loads in flight than long rows in one warp,
// and idle threads cost issue slots: 12800 rows of 2304 to 8 bits take 43 us
// on 96 threads with 3 units each, 47 - 49 on 128 (a quarter of the units past
// the end), 53 on a warp with 10 units.
template <typename T, int kMode, int NV, int TPR>
__global__ void __launch_bounds__(TPR <= 32 ? 128 : TPR) rms_norm_kernel(const NormParams p) {
  constexpr int kRowsCta = TPR <= 32 ? 128 / TPR : 1, VEC = kMode == kNormOne ? 1 : 8;
  __shared__ float part[TPR < 32 ? 1 : TPR / 32];
  const int t = threadIdx.x % TPR;
  const int row = static_cast<int>(blockIdx.x * kRowsCta + threadIdx.x / TPR);  // below 2^31
  // rows past the last take part in the shuffles as zeros; those that fill the
  // last scale tile up write their scales, zeros too
  const bool live = row < p.rows;
  int xr = 0, rr = 0, hr = 0;
  const bool found = live && norm_rows(p, row, t == 0, xr, rr, hr);
  const T* x = static_cast<const T*>(p.x) + static_cast<size_t>(found ? xr : 0) * p.D;
  const T* res = p.res != nullptr ? static_cast<const T*>(p.res) + static_cast<size_t>(found ? rr : 0) * p.D : nullptr;
  T* h = p.h != nullptr ? static_cast<T*>(p.h) + static_cast<size_t>(found ? hr : p.h_full || !live ? 0 : row) * p.D : nullptr;
  T* y = p.y != nullptr ? static_cast<T*>(p.y) + static_cast<size_t>(live ? row : 0) * p.D : nullptr;
  const bool h_found = p.h != nullptr && (found || (live && !p.h_full));
  // first element of unit u (shifted: of the row's first whole unit or before), units
  const int shift = kMode == kNormShift ? (row & 7) * (p.D & 7) & 7 : 0;
  const int units = kMode == kNormOne ? p.D : (p.D + shift + 7) / 8;
  // elements of the tensor from the row's first on
  const long long left = kMode == kNormShift ? static_cast<long long>(p.rows - row) * p.D : 0;

  float v[NV * VEC];
  if constexpr (kMode == kNormOne) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = i * TPR + t;
      v[i] = found && u < units ? to_float(x[u]) : 0.f;
    }
    if (res != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int u = i * TPR + t;
        if (found && u < units) v[i] += to_float(res[u]);
      }
    }
  } else {
    auto load = [&](Raw8<T>& r, const T* f, int u) {
      r.zero();
      if (!found || u >= units) return;
      if (kMode == kNormVec || 8 * u - shift + 8 <= left) {
        r.load(f + (8 * u - shift));
      } else {  // the tensor ends inside this unit
        T* e = reinterpret_cast<T*>(&r);
        for (int k = 0; k < 8; ++k)
          if (8 * u - shift + k >= 0 && 8 * u - shift + k < p.D) e[k] = f[8 * u - shift + k];
      }
    };
    Raw8<T> a[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) load(a[i], x, i * TPR + t);
    if (res != nullptr) {
      Raw8<T> b[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) load(b[i], res, i * TPR + t);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8];
        a[i].get(v + 8 * i);
        b[i].get(f);
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          f2_unpack(f2_add(f2_pack(v[8 * i + e], v[8 * i + e + 1]), f2_pack(f[e], f[e + 1])), v[8 * i + e],
                    v[8 * i + e + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) a[i].get(v + 8 * i);
    }
    if constexpr (kMode == kNormShift) {  // the neighbouring rows' elements
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = 8 * (i * TPR + t) - shift + e;
          if (at < 0 || at >= p.D) v[8 * i + e] = 0.f;
        }
    }
  }
  // (kNormShift: without S)
  const bool ok = kMode == kNormShift ? found : live && norm_in_order(p, row, t == 0) && found;
  const bool h_write = kMode == kNormShift ? h_found : h_found && (ok || !p.h_full);
  float ss = 0.f;
  if constexpr (VEC == 8) {
    uint64_t s2 = f2_pack(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV * 8; i += 2) {
      const uint64_t x2 = f2_pack(v[i], v[i + 1]);
      s2 = f2_fma(x2, x2, s2);
    }
    float lo, hi;
    f2_unpack(s2, lo, hi);
    ss = lo + hi;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) ss = fmaf(v[i], v[i], ss);
  }
  ss = row_sum<TPR>(ss, part);
  const float rstd = ok ? 1.f / sqrtf(fmaf(ss, p.inv_D, p.eps)) : 0.f;

#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int u = i * TPR + t;
    const bool in = u < units;
    if constexpr (kMode == kNormOne) {
      if (in) {
        if (h_write) h[u] = from_float<T>(v[i]);
        const float f = ok ? (p.w != nullptr ? v[i] * rstd * __ldg(p.w + u) : v[i] * rstd) : 0.f;
        if (y != nullptr && live) y[u] = from_float<T>(f);
      }
      continue;
    } else {
      float f[8];
      scale8(v + 8 * i, rstd, f);
      const int at = 8 * u - shift;  // the unit's first element
      if (kMode == kNormVec || (at >= 0 && at + 8 <= p.D)) {
        if (in && h_write) store8(h + at, v + 8 * i);
        if (in && p.w != nullptr) {
          if constexpr (kMode == kNormVec) {
            const float4 w0 = __ldg(reinterpret_cast<const float4*>(p.w) + 2 * u);
            const float4 w1 = __ldg(reinterpret_cast<const float4*>(p.w) + 2 * u + 1);
            f2_unpack(f2_mul(f2_pack(f[0], f[1]), f2_pack(w0.x, w0.y)), f[0], f[1]);
            f2_unpack(f2_mul(f2_pack(f[2], f[3]), f2_pack(w0.z, w0.w)), f[2], f[3]);
            f2_unpack(f2_mul(f2_pack(f[4], f[5]), f2_pack(w1.x, w1.y)), f[4], f[5]);
            f2_unpack(f2_mul(f2_pack(f[6], f[7]), f2_pack(w1.z, w1.w)), f[6], f[7]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= __ldg(p.w + at + e);
          }
        }
        if (!ok) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = 0.f;
        }
        if (in && live && y != nullptr) store8(y + at, f);
      } else if (in && live) {  // an edge of the row
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at + e >= 0 && at + e < p.D) {
            if (h_write) h[at + e] = from_float<T>(v[8 * i + e]);
            if (y != nullptr) y[at + e] = from_float<T>(ok ? (p.w != nullptr ? f[e] * __ldg(p.w + at + e) : f[e]) : 0.f);
          }
      }
      if constexpr (kMode == kNormVec && TPR >= 16) {
        if (p.q != nullptr) {
          // blocks of 32: four threads; a word of scales: sixteen (D is a
          // multiple of 32, so a block is inside the row or past its end)
          float top = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(f[e]));
          uint32_t amax = __float_as_uint(top);
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          float inv;
          uint32_t word = e8m0_scale<8>(amax, inv);
          if (!in) word = 0;
          word <<= 8 * ((t >> 2) & 3);
          word |= __shfl_xor_sync(0xffffffffu, word, 4);
          word |= __shfl_xor_sync(0xffffffffu, word, 8);
          if (in && row < p.rows_pad) {
            if (live)
              *reinterpret_cast<uint2*>(p.q + static_cast<size_t>(row) * p.D + u * 8) =
                  e4m3x8(f, inv);
            if ((t & 15) == 0) *reinterpret_cast<uint32_t*>(p.q_scales + mx_scale_at(row, u >> 2, p.ct)) = word;
          }
        }
      }
    }
  }
}

// Rows too long for the registers: 512 threads read the row twice. In place
// each element is read and written by one thread, in this order.
template <typename T>
__global__ void __launch_bounds__(512) rms_norm_long_kernel(const NormParams p) {
  __shared__ float part[16];
  const int row = static_cast<int>(blockIdx.x);
  int xr, rr, hr;
  const bool found = norm_rows(p, row, threadIdx.x == 0, xr, rr, hr);
  const bool ok = norm_in_order(p, row, threadIdx.x == 0) && found;
  const T* x = static_cast<const T*>(p.x) + static_cast<size_t>(ok ? xr : 0) * p.D;
  const T* res = p.res != nullptr ? static_cast<const T*>(p.res) + static_cast<size_t>(ok ? rr : 0) * p.D : nullptr;
  T* h = p.h != nullptr ? static_cast<T*>(p.h) + static_cast<size_t>(ok ? hr : p.h_full ? 0 : row) * p.D : nullptr;
  const bool h_write = p.h != nullptr && (ok || !p.h_full);
  T* y = p.y != nullptr ? static_cast<T*>(p.y) + static_cast<size_t>(row) * p.D : nullptr;
  float ss = 0.f;
  if (ok)
    for (int u = threadIdx.x; u < p.D; u += 512) {
      float v = to_float(x[u]);
      if (res != nullptr) v += to_float(res[u]);
      ss = fmaf(v, v, ss);
    }
  ss = row_sum<512>(ss, part);
  const float rstd = ok ? 1.f / sqrtf(fmaf(ss, p.inv_D, p.eps)) : 0.f;
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
