// rope.cuh - rotary positions of the queries and keys.
//
// Pair i of a head turns by the angle pos * f_i:
//     (a, b) -> m (a cos - b sin, b cos + a sin)
// with (a, b) = (x[i], x[i + r/2]) (halves) or (x[2i], x[2i + 1])
// (interleaved); elements from r on pass through. On a latent grid the pairs
// are shared out over the axes, each with a position of its own.
//
// Angles: a frequency is held as a fraction of a turn in 64-bit fixed
// point, F = f / (2 pi) 2^64. pos * F modulo 2^64 is then the phase modulo a
// turn with no loss at any position: the integer product drops whole turns
// by itself. Its top 32 bits go to sincospi as a float in [-1, 1).
#pragma once

#include "mx_quant.cuh"

namespace safe {

struct RopeTensor {
  const void* x;
  void* o;
  long long xb, xn, xh;  // strides in elements: sample, row, head (the head dim is contiguous)
  long long ob, on, oh;
  int H;
};

struct RopeParams {
  RopeTensor t[2];        // queries, keys (H = 0: none)
  const long long* freq;  // [r / 2] turns of one position in 2^-64
  const int32_t* pos;     // [N, axes] or [B, N, axes] (pos_b = elements of a sample, 0: shared), or null: the token index
  long long pos_b;
  const int32_t* S;       // [B, R] tokens of the rows, or null
  int axes, sec0, sec1;   // pairs of the first and second axis (the others belong to the third)
  int N, R, d, r;
  float m;
  long long rows;         // B * R
  int copy_tail;          // elements r .. d have to be copied (0: in place)
};

constexpr int kRopeWarps = 4;

// A warp takes a token: it computes the r / 2 rotations once (shared memory),
// then turns all heads of both tensors. Bound by memory: q and k are read and
// written once. VEC: 8 elements for each access (16-byte aligned rows and heads,
// whole units), else single pairs.
template <typename T, bool kPairs, bool kVec>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const RopeParams p) {
  extern __shared__ float2 rope_cs[];  // [warps][r / 2] cos, sin
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = p.r / 2;
  const long long row = static_cast<long long>(blockIdx.x) * kRopeWarps + warp;
  if (row >= p.rows) return;
  float2* cs = rope_cs + warp * ((half + 3) & ~3);
  const long long b = row / p.R, r = row - b * p.R;
  long long token = r;
  if (p.S != nullptr) {
    token = __ldg(p.S + row);
    if (token < 0 || token >= p.N) {  // flagged; the row turns as token 0
      if (lane == 0) raise_status(1 << 5);
      token = 0;
    }
  }
  const int32_t* pos = p.pos != nullptr ? p.pos + b * p.pos_b + token * p.axes : nullptr;
  for (int i = lane; i < half; i += 32) {
    const int axis = i < p.sec0 ? 0 : i < p.sec0 + p.sec1 ? 1 : 2;
    const long long at = pos != nullptr ? __ldg(pos + axis) : token;
    const unsigned long long phase = static_cast<unsigned long long>(at) * static_cast<unsigned long long>(__ldg(p.freq + i));
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    cs[i] = make_float2(c * p.m, s * p.m);
  }
  __syncwarp();
  for (int k = 0; k < 2; ++k) {
    const RopeTensor& t = p.t[k];
    if (t.H == 0) continue;
    const T* x = static_cast<const T*>(t.x) + b * t.xb + r * t.xn;
    T* o = static_cast<T*>(t.o) + b * t.ob + r * t.on;
    if constexpr (kVec) {
      // units of a head: halves: r / 16 of 8 pairs; interleaved: r / 8 of 4 pairs; then the tail's (d - r) / 8
      const int rot = kPairs ? p.r / 8 : p.r / 16, per = rot + (p.copy_tail ? (p.d - p.r) / 8 : 0);
      for (int u = lane; u < t.H * per; u += 32) {
        const int head = u / per, c = u - head * per;
        const T* xh = x + head * t.xh;
        T* oh = o + head * t.oh;
        Raw8<T> ra, rb;
        float a[8], bb[8];
        if (c < rot) {
          if constexpr (kPairs) {
            ra.load(xh + 8 * c);
            ra.get(a);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 w = cs[4 * c + e];
              bb[2 * e] = a[2 * e] * w.x - a[2 * e + 1] * w.y;
              bb[2 * e + 1] = a[2 * e + 1] * w.x + a[2 * e] * w.y;
            }
            store8(oh + 8 * c, bb);
          } else {
            ra.load(xh + 8 * c);
            rb.load(xh + half + 8 * c);
            ra.get(a);
            rb.get(bb);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 w = cs[8 * c + e];
              const float f = a[e] * w.x - bb[e] * w.y;
              bb[e] = bb[e] * w.x + a[e] * w.y;
              a[e] = f;
            }
            store8(oh + 8 * c, a);
            store8(oh + half + 8 * c, bb);
          }
        } else {
          const int e = p.r + 8 * (c - rot);
          ra.load(xh + e);
          ra.get(a);
          store8(oh + e, a);
        }
      }
    } else {
      const int per = half + (p.copy_tail ? p.d - p.r : 0);
      for (int u = lane; u < t.H * per; u += 32) {
        const int head = u / per, c = u - head * per;
        const T* xh = x + head * t.xh;
        T* oh = o + head * t.oh;
        if (c < half) {
          const int i = kPairs ? 2 * c : c, j = kPairs ? 2 * c + 1 : c + half;
          const float a = to_float(xh[i]), bb = to_float(xh[j]);
          const float2 w = cs[c];
          oh[i] = from_float<T>(a * w.x - bb * w.y);
          oh[j] = from_float<T>(bb * w.x + a * w.y);
        } else {
          oh[p.r + c - half] = xh[p.r + c - half];
        }
      }
    }
  }
}

}  // namespace safe
