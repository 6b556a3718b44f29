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
  uint32_t rows;          // B * R
  int copy_tail;          // elements r .. d have to be copied (0: in place)
  int warps;              // warps of a token (rope_vec_kernel)
};

constexpr int kRopeWarps = 4;

// Token of a row, and where its positions are (null: the token is the position).
__device__ __forceinline__ const int32_t* rope_token(const RopeParams& p, uint32_t row, uint32_t b, uint32_t r, int lane,
                                                     int& token) {
  token = static_cast<int>(r);
  if (p.S != nullptr) {
    token = __ldg(p.S + row);
    if (token < 0 || token >= p.N) {  // flagged; the row turns as token 0
      if (lane == 0) raise_status(1 << 5);
      token = 0;
    }
  }
  return p.pos != nullptr ? p.pos + b * p.pos_b + static_cast<long long>(token) * p.axes : nullptr;
}

// (m cos, m sin) of pair i at a position.
__device__ __forceinline__ float2 rope_rotation(const RopeParams& p, int i, long long at) {
  const unsigned long long phase = static_cast<unsigned long long>(at) * static_cast<unsigned long long>(__ldg(p.freq + i));
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
  return make_float2(c * p.m, s * p.m);
}
__device__ __forceinline__ int rope_axis(const RopeParams& p, int i) {
  return i < p.sec0 ? 0 : i < p.sec0 + p.sec1 ? 1 : 2;
}

// Turns 8 pairs: a and v hold pairs (e, e) (halves) or 4 neighbouring pairs each.
template <bool kPairs>
__device__ __forceinline__ void rope_turn(float* a, float* v, const float2* w) {
  if constexpr (kPairs) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float f = a[2 * e], k = v[2 * e];
      a[2 * e] = f * w[e].x - a[2 * e + 1] * w[e].y;
      a[2 * e + 1] = a[2 * e + 1] * w[e].x + f * w[e].y;
      v[2 * e] = k * w[e + 4].x - v[2 * e + 1] * w[e + 4].y;
      v[2 * e + 1] = v[2 * e + 1] * w[e + 4].x + k * w[e + 4].y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = a[e];
      a[e] = f * w[e].x - v[e] * w[e].y;
      v[e] = v[e] * w[e].x + f * w[e].y;
    }
  }
}

// The r / 2 rotations of a token (m cos, m sin), by `n` threads.
__device__ __forceinline__ void rope_rotations(const RopeParams& p, const int32_t* pos, int token, int t, int n,
                                               float2* cs) {
  for (int i = t; i < p.r / 2; i += n) cs[i] = rope_rotation(p, i, pos != nullptr ? __ldg(pos + rope_axis(p, i)) : token);
}

// p.warps warps (1, 2 or 4) take a token: they compute the rotations once, in
// shared memory, while the heads' elements are on their way, then turn all
// heads of both tensors. A lane keeps one unit of 16 elements (8 pairs, their
// rotations in registers) and walks the heads with it, U at a time: `per` =
// r / 16 lanes share a head, 32 / per heads go side by side. As many warps
// share a token as make its heads one batch of loads each: one latency from
// start to end, for few tokens. For 16-byte aligned rows and heads, r a
// multiple of 16, d of 8.
template <typename T, bool kPairs, int U>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_vec_kernel(const RopeParams p) {
  extern __shared__ float4 rope_cs4[];  // [tokens of the CTA][r / 2] cos, sin
  const int lane = threadIdx.x & 31, half = p.r / 2;
  const int slot = (threadIdx.x >> 5) / p.warps, part = (threadIdx.x >> 5) - slot * p.warps;
  const uint32_t at = blockIdx.x * (kRopeWarps / p.warps) + slot;
  const bool live = at < p.rows;  // the last CTA's spare warps repeat its last token, without stores
  const uint32_t row = live ? at : p.rows - 1;
  float2* cs = reinterpret_cast<float2*>(rope_cs4) + slot * half;  // half is a multiple of 8
  const uint32_t b = row / static_cast<uint32_t>(p.R), r = row - b * p.R;
  int token;
  const int32_t* pos = rope_token(p, row, b, r, part == 0 ? lane : 1, token);
  const T* xq = static_cast<const T*>(p.t[0].x) + b * p.t[0].xb + r * p.t[0].xn;
  T* oq = static_cast<T*>(p.t[0].o) + b * p.t[0].ob + r * p.t[0].on;
  const T* xk = static_cast<const T*>(p.t[1].x) + b * p.t[1].xb + r * p.t[1].xn;
  T* ok = static_cast<T*>(p.t[1].o) + b * p.t[1].ob + r * p.t[1].on;
  const int Hq = p.t[0].H, H = Hq + p.t[1].H;
  auto from = [&](int h) { return h < Hq ? xq + h * p.t[0].xh : xk + (h - Hq) * p.t[1].xh; };
  auto to = [&](int h) { return h < Hq ? oq + h * p.t[0].oh : ok + (h - Hq) * p.t[1].oh; };

  const int per = p.r / 16, side = per < 32 ? 32 / per : 1;
  const int g = per < 32 ? lane / per : 0, c0 = per < 32 ? lane - g * per : lane;
  Raw8<T> x[U], y[U];
  auto load = [&](int h, int c) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * side < H) {
        const T* f = from(h + u * side);
        x[u].load(f + (kPairs ? 16 * c : 8 * c));
        y[u].load(f + (kPairs ? 16 * c + 8 : half + 8 * c));
      }
  };
  const int first = live && g < side && c0 < per ? g + part * U * side : H;  // the lanes left over take no head
  load(first, c0);
  rope_rotations(p, pos, token, part * 32 + lane, 32 * p.warps, cs);
  __syncthreads();
  for (int c = c0; c < per; c += 32) {
    float2 w[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 f = reinterpret_cast<const float4*>(cs)[4 * c + e];
      w[2 * e] = make_float2(f.x, f.y);
      w[2 * e + 1] = make_float2(f.z, f.w);
    }
    for (int h = first; h < H; h += U * side * p.warps) {
      if (h != first || c != c0) load(h, c);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * side < H) {
          float a[8], v[8];
          x[u].get(a);
          y[u].get(v);
          rope_turn<kPairs>(a, v, w);
          T* o = to(h + u * side);
          store8(o + (kPairs ? 16 * c : 8 * c), a);
          store8(o + (kPairs ? 16 * c + 8 : half + 8 * c), v);
        }
    }
  }
  if (!p.copy_tail || !live) return;
  const int tail = (p.d - p.r) / 8, tside = tail < 32 ? 32 / tail : 1;  // units of 8
  const int tg = tail < 32 ? lane / tail : 0;
  if (tg >= tside) return;
  for (int c = tail < 32 ? lane - tg * tail : lane; c < tail; c += 32)
    for (int h = tg + part * U * tside; h < H; h += U * tside * p.warps) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * tside < H) x[u].load(from(h + u * tside) + p.r + 8 * c);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * tside < H) x[u].store(to(h + u * tside) + p.r + 8 * c);
    }
}

// Many tokens whose heads lie together in their rows: persistent CTAs copy whole
// rows into a ring of shared memory, turn them there and copy them back, all
// by asynchronous bulk copies, so that reads and writes go in whole lines and
// stay ahead of the arithmetic whatever the head dim is. (With plain loads the
// 96-byte halves of a head of 96 measured 172 - 190 us at 51200 tokens of
// 24 + 24 heads, bf16; this 152.) Token i of the CTA uses stage i % kRopeStages:
// two tokens are on their way in and two on their way out.
constexpr int kRopeStages = 4;
constexpr int kRopeBulkMax = 27 * 1024;  // bytes of a token's rows: two CTAs an SM
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
// All but the thread's last bulk group have read their shared memory.
__device__ __forceinline__ void bulk_wait_read_but_one() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

template <typename T, bool kPairs>
__global__ void __launch_bounds__(128) rope_bulk_kernel(const RopeParams p) {
  extern __shared__ __align__(128) uint8_t rope_sm[];  // [stages][row bytes of q and k], [2][r / 2] cos, sin, barriers
  const int tid = threadIdx.x, half = p.r / 2;
  const uint32_t qb = p.t[0].H * p.d * sizeof(T), kb = p.t[1].H * p.d * sizeof(T);  // multiples of 16
  const uint32_t stage = (qb + kb + 127) & ~127u;
  float2* cs = reinterpret_cast<float2*>(rope_sm + kRopeStages * stage);
  uint64_t* full = reinterpret_cast<uint64_t*>(cs + 2 * half);
  __shared__ int abort_flag;
  const uint32_t n = p.rows > blockIdx.x ? (p.rows - 1 - blockIdx.x) / gridDim.x + 1 : 0;
  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < kRopeStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  auto load = [&](uint32_t i) {  // thread 0
    const uint32_t row = blockIdx.x + i * gridDim.x, b = row / static_cast<uint32_t>(p.R), r = row - b * p.R;
    uint64_t* bar = &full[i % kRopeStages];
    const uint32_t dst = smem_u32(rope_sm + (i % kRopeStages) * stage);
    mbar_arrive_expect_tx(bar, qb + kb);
    bulk_load(dst, static_cast<const T*>(p.t[0].x) + b * p.t[0].xb + r * p.t[0].xn, qb, bar);
    if (kb) bulk_load(dst + qb, static_cast<const T*>(p.t[1].x) + b * p.t[1].xb + r * p.t[1].xn, kb, bar);
  };
  auto rotations = [&](uint32_t i) {
    const uint32_t row = blockIdx.x + i * gridDim.x, b = row / static_cast<uint32_t>(p.R);
    int token;
    const int32_t* pos = rope_token(p, row, b, row - b * p.R, tid, token);
    rope_rotations(p, pos, token, tid, 128, cs + (i & 1) * half);
  };
  if (tid == 0)
    for (uint32_t i = 0; i < kRopeStages - 2 && i < n; ++i) load(i);
  if (n > 0) rotations(0);
  __syncthreads();

  const int per = p.r / 16, side = per < 128 ? 128 / per : 1;
  const int g = tid / per, c = tid - g * per, H = p.t[0].H + p.t[1].H;  // r <= 1024: per <= 64
  uint32_t i = 0;
  for (; i < n; ++i) {
    if (tid == 0 && i + kRopeStages - 2 < n) {
      bulk_wait_read_but_one();  // token i - 2 has left the stage
      load(i + kRopeStages - 2);
    }
    bool ok = mbar_wait(&full[i % kRopeStages], (i / kRopeStages) & 1, &abort_flag);
    if (ok && g < side) {
      float2 w[8];
      const float4* f = reinterpret_cast<const float4*>(cs + (i & 1) * half) + 4 * c;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[2 * e] = make_float2(f[e].x, f[e].y);
        w[2 * e + 1] = make_float2(f[e].z, f[e].w);
      }
      T* rowp = reinterpret_cast<T*>(rope_sm + (i % kRopeStages) * stage);
      for (int h = g; h < H; h += side) {
        T* x = rowp + h * p.d + (kPairs ? 16 * c : 8 * c);
        T* y = x + (kPairs ? 8 : half);
        Raw8<T> rx, ry;
        float a[8], v[8];
        rx.load(x);
        ry.load(y);
        rx.get(a);
        ry.get(v);
        rope_turn<kPairs>(a, v, w);
        store8(x, a);
        store8(y, v);
      }
    }
    if (i + 1 < n) rotations(i + 1);
    fence_proxy_async_smem();
    if (__syncthreads_or(!ok)) break;
    if (tid == 0) {
      const uint32_t row = blockIdx.x + i * gridDim.x, b = row / static_cast<uint32_t>(p.R), r = row - b * p.R;
      const uint32_t src = smem_u32(rope_sm + (i % kRopeStages) * stage);
      bulk_store(static_cast<T*>(p.t[0].o) + b * p.t[0].ob + r * p.t[0].on, src, qb);
      if (kb) bulk_store(static_cast<T*>(p.t[1].o) + b * p.t[1].ob + r * p.t[1].on, src + qb, kb);
      bulk_commit_group();
    }
  }
  if (tid == 0) {
    bulk_wait_read_all();
    // given up: let the copies on their way in land before the CTA ends
    for (uint32_t j = i; i < n && j < n && j < i + kRopeStages - 1; ++j) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&full[j % kRopeStages], (j / kRopeStages) & 1) && globaltimer_ns() - t0 < 200000000ull) {
      }
    }
  }
}

// The same for any strides, alignment and r: a lane turns single pairs, one load
// and one store of an element at a time (51200 tokens of 24 + 24 heads of 96,
// bf16, in rows 2 bytes off: 391 us; with r = 20: 580; aligned with r = 96, from a
// fused projection: 166).
template <typename T, bool kPairs>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const RopeParams p) {
  extern __shared__ float4 rope_cs4[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = p.r / 2;
  const uint32_t row = blockIdx.x * kRopeWarps + warp;
  if (row >= p.rows) return;
  float2* cs = reinterpret_cast<float2*>(rope_cs4) + warp * half;
  const uint32_t b = row / static_cast<uint32_t>(p.R), r = row - b * p.R;
  int token;
  const int32_t* pos = rope_token(p, row, b, r, lane, token);
  rope_rotations(p, pos, token, lane, 32, cs);
  __syncwarp();
  for (int k = 0; k < 2; ++k) {
    const RopeTensor& t = p.t[k];
    if (t.H == 0) continue;
    const T* x = static_cast<const T*>(t.x) + b * t.xb + r * t.xn;
    T* o = static_cast<T*>(t.o) + b * t.ob + r * t.on;
    const int per = half + (p.copy_tail ? p.d - p.r : 0);
    for (int u = lane; u < t.H * per; u += 32) {
      const int head = u / per, c = u - head * per;
      const T* xh = x + head * t.xh;
      T* oh = o + head * t.oh;
      if (c < half) {
        const int i = kPairs ? 2 * c : c, j = kPairs ? 2 * c + 1 : c + half;
        const float a = to_float(xh[i]), v = to_float(xh[j]);
        const float2 w = cs[c];
        oh[i] = from_float<T>(a * w.x - v * w.y);
        oh[j] = from_float<T>(v * w.x + a * w.y);
      } else {
        oh[p.r + c - half] = xh[p.r + c - half];
      }
    }
  }
}

}  // namespace safe
