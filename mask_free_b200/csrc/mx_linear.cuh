// mx_linear.cuh - row-wise layers of the row-selective block with microscaled operands.
//
//     Y[r, :] = act( alpha * sum_c X[r, c] W[:, c] + bias )
// X and W are microscaled matrices (mx_quant.cuh) of the same format; the
// tensor core multiplies the 8- or 4-bit elements, applies both block scales
// to each block's products and adds in fp32 (tcgen05.mma .block_scale).
//
// linear_pair_kernel's structure with other operands: a CTA pair computes
// 256 x 256 output tiles, each CTA 128 rows. A stage of the ring is 128
// bytes of every row (128 e4m3 or 256 e2m1 elements, four MMA steps of 32
// bytes) with the scales that belong to them:
//   A, B     128 rows x 128 B each: the CTA's rows of X and its half of the W rows
//   scale A  of the CTA's own rows (one scale tile for each 4 scales of a row)
//   scale B  of all 256 W rows, in both CTAs
// Scales travel shared memory -> TMEM by tcgen05.cp (32 lanes x 16 B, copied
// to all four lane quarters) right before the MMAs that use them. A copy is
// ordered before the MMAs behind it; that it stays behind the MMAs in front,
// whose scales it would overwrite, nothing says. So stages take two scale
// buffers in turn, and a warp of its own keeps a stage from the issuing
// warp until the MMAs two stages back are complete: it holds the second of the
// two arrivals that the stage's barrier counts. (With one buffer and no wait 303
// us, so 304: nvfp4 51200 x 2304 x 6912; with the wait in the issuing warp 344,
// whatever stage it waits for.)
// TMEM (512 columns): the last 96 hold the scales; the two accumulators of
// 256 columns (tile i uses i & 1) overlap in 96 columns in the middle, the last
// of accumulator 0 and the first of 1. A tile's first MMA waits until the
// epilogue has read these from the tile before (with the 32 columns that its
// warps read beside them); the others are read while the next tile is multiplied.
// Every MMA of a tile has the same shape and accumulator: consecutive ones of one
// thread are ordered under that condition only (a form whose first and last
// stages did the shared columns apart, to hide that wait, added to them in two
// shapes; with a wait for completion wherever the shape changes it was slower
// than this one, as was that with both shapes in every stage: nvfp4
// 51200 x 2304 x 6912 336 and 328 us against 301).
//
// What bounds it: a stage is 34 - 38 KB into shared memory and as much out of
// it for 512 cycles of MMA, and 1000 W. A call by itself after an L2 flush
// (PFLOP/s; 51200 rows at d_in = 2304, 12800 at 9216, d_out 6912): nvfp4 5.1 - 5.4
// and 6.2, mxfp4 5.5 and 6.7, mxfp8 2.9 and 2.7; calls back to back for two
// seconds, when power sets the clock: nvfp4 4.1 and 5.0, mxfp4 4.3 and 5.4, mxfp8
// 2.3 and 2.2. Measured on the way, each at its time (nvfp4): tiles of 192 columns with accumulators apart 4.2 / 4.9; the
// output through shared memory and tiled stores, which compete with the
// operands, 4.9 / 5.8 against 5.2 / 6.2; a release instead of a relaxed arrival
// for the accumulator 4.8 / 6.1.
#pragma once

#include "linear.cuh"
#include "mx_quant.cuh"

namespace safe {

// Instruction descriptor of the block-scaled kinds: element and scale formats,
// shape, which byte of a scale word the step takes.
__host__ __device__ constexpr uint32_t make_idesc_mx(int fmt, int M, int N, int sf_id) {
  return (static_cast<uint32_t>(sf_id) << 4)                   // scale B byte
         | ((fmt == kMxFp8 ? 0u : 1u) << 7)                    // A: e4m3 = 0 (mxf8f6f4), e2m1 = 1 (mxf4)
         | ((fmt == kMxFp8 ? 0u : 1u) << 10)                   // B
         | (static_cast<uint32_t>(N >> 3) << 17)               // N / 8
         | ((fmt == kNvFp4 ? 0u : 1u) << 23)                   // scales: e4m3 = 0, e8m0 = 1
         | (static_cast<uint32_t>(M >> 7) << 27)               // M / 128
         | (static_cast<uint32_t>(sf_id) << 29);               // scale A byte
}

template <int kFmt>
__device__ __forceinline__ void umma_pair_mx_if(uint32_t leader, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (kFmt == kNvFp4) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
            "r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(leader)
        : "memory");
  } else if constexpr (kFmt == kMxFp4) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(leader)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
            "r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(leader)
        : "memory");
  }
}

// tma_load_2d_pair for a warp-uniform code path: the lane with `leader` != 0 issues.
__device__ __forceinline__ void tma_load_2d_pair_if(uint32_t leader, uint32_t dst, const CUtensorMap* map, uint32_t mbar,
                                                    int c0, int c1) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(c0), "r"(c1), "r"(leader)
      : "memory");
}
// mbar_arrive_cluster without its release: for a barrier that only hands tensor
// memory back, which the arriving warp has read (tcgen05.wait::ld). A
// release waits for the warp's stores of the last tile, 1100 cycles here.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t caddr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}
// umma_pair_commit_if on the barrier at shared-memory address `bar` of both CTAs.
__device__ __forceinline__ void umma_pair_commit_both_if(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %2, 0;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"(static_cast<uint16_t>(3)), "r"(leader)
      : "memory");
}
// warp_wait for waits that are short as a rule: the clock is read only after
// some polls in vain.
__device__ __forceinline__ bool warp_wait_short(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, abort);
}

// 32 bytes to memory (32-byte aligned).
__device__ __forceinline__ void st_global32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// One scale tile (512 B of each CTA's shared memory, at the same offset) into
// four TMEM columns of each CTA of the pair.
__device__ __forceinline__ void tmem_copy_scales_pair_if(uint32_t leader, uint32_t taddr, uint64_t sdesc) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %2, 0;\n\t"
      "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(sdesc), "r"(leader)
      : "memory");
}

constexpr int kMxPieces = 96;  // pieces at most

struct MxLinearParams {
  CUtensorMap x_map;   // bytes [M, row bytes], box 128 x 128, 128B swizzle
  CUtensorMap w_map;   // bytes [d_out, row bytes], box 128 x 128, 128B swizzle
  CUtensorMap xs_map;  // scale tiles as 8-byte words [row blocks, tiles * 64], box (tiles of a stage * 64) x 1
  CUtensorMap ws_map;  // the same of W, box (tiles of a stage * 64) x 2
  const float* bias;   // [d_out] or null
  __nv_bfloat16* Y;    // [M, d_out]
  float alpha;
  int M, row_bytes, d_out, act;
  int n_tiles;         // column tiles
  int wide;            // rows of Y are 32-byte aligned
  // Units of work: the first `whole` tiles, then pieces along d_in of the other
  // tiles, whose sums go to `part` [piece][256][256] fp32. A table, not a
  // division: its entries are uniform constants to the compiler, as all
  // operands of the issue loop have to be. (Where it cannot prove that, it
  // guards every MMA, copy and barrier instruction against lanes that
  // disagree, and the loop costs more than the MMAs: 313 us instead of 262,
  // nvfp4, 12800 x 9216 x 6912.)
  int whole, units;
  float* part;
  uint16_t piece_tile[kMxPieces], piece_k0[kMxPieces], piece_n[kMxPieces];  // tile, first stage, stages (8192 at most)
};

constexpr int kMxThreads = 640;  // warps 0-3 producers / MMA / TMEM, warps 4-19 epilogue
constexpr int kMxTileN = 256;
constexpr int kMxABytes = 128 * 128, kMxBBytes = 128 * 128;
// scale tiles along a row in a stage: 128 B hold 4 (mxfp8), 8 (mxfp4) or 16 (nvfp4) scales
__host__ __device__ constexpr int mx_stage_tiles(int fmt) { return fmt == kMxFp8 ? 1 : fmt == kMxFp4 ? 2 : 4; }
__host__ __device__ constexpr int mx_stage_bytes(int fmt) { return kMxABytes + kMxBBytes + 3 * 512 * mx_stage_tiles(fmt); }
// As many stages as fit (5 of nvfp4, 6 of the others).
__host__ __device__ constexpr int mx_stages(int fmt) { return (227 * 1024 - 1024 - 16 * 256 - 256) / mx_stage_bytes(fmt); }
__host__ __device__ constexpr int mx_linear_smem(int fmt) {
  return 1024 + mx_stages(fmt) * mx_stage_bytes(fmt) + 16 * 256 + 256;
}

// GELU in its tanh form of two values: x / (1 + 2^t), t = x (c1 + c2 x^2) with
// c1 = -2 sqrt(2 / pi) / ln 2 and c2 = 0.044715 c1 (see gelu_tanh_f), in packed
// arithmetic: 11 instructions with the rounding, 4 of them the exp unit's. (One
// reciprocal for both, of the product, takes one of those less, but 19 with
// what keeps the product finite and a NaN to itself: nvfp4, 12800 x 2304 x 9216,
// back to back 158 us at that step, this 149. Now 125, without an activation 114,
// in 60 calls back to back.)
__device__ __forceinline__ uint64_t gelu_tanh_2(uint64_t x) {
  const uint64_t c2 = f2_pack(-0.10294324f, -0.10294324f), c1 = f2_pack(-2.3022082f, -2.3022082f);
  float t0, t1, a, b;
  f2_unpack(f2_mul(x, f2_fma(f2_mul(x, x), c2, c1)), t0, t1);
  f2_unpack(f2_add(f2_pack(ex2_approx(t0), ex2_approx(t1)), f2_pack(1.f, 1.f)), a, b);
  return f2_mul(x, f2_pack(rcp_approx(a), rcp_approx(b)));
}

// act(alpha v + bias) of a row's next 64 columns (of which `left` exist), rounded
// to bf16, to memory: stores of 32 bytes (whole sectors) where rows are so
// aligned, else of 16. Every lane reads all 64 biases from shared memory, in
// single words: vectors that all lanes read at once took six passes each, 1 - 3 %
// of a call.
template <bool kGelu>
__device__ __forceinline__ void mx_store_row(const uint32_t* v, float alpha, uint32_t bias, __nv_bfloat16* y, int left,
                                             int wide) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {  // 16 columns
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t at = bias + 4 * (16 * c + 4 * k);
      float4 b;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(b.x) : "r"(at));
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(b.y) : "r"(at + 4));
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(b.z) : "r"(at + 8));
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(b.w) : "r"(at + 12));
      const uint64_t al = f2_pack(alpha, alpha);
      const uint32_t* vk = v + 16 * c + 4 * k;
      uint64_t f0 = f2_fma(f2_pack(__uint_as_float(vk[0]), __uint_as_float(vk[1])), al, f2_pack(b.x, b.y));
      uint64_t f1 = f2_fma(f2_pack(__uint_as_float(vk[2]), __uint_as_float(vk[3])), al, f2_pack(b.z, b.w));
      if constexpr (kGelu) {
        f0 = gelu_tanh_2(f0);
        f1 = gelu_tanh_2(f1);
      }
      float y0, y1, y2, y3;
      f2_unpack(f0, y0, y1);
      f2_unpack(f1, y2, y3);
      w[2 * k] = pack_bf16x2(y0, y1);
      w[2 * k + 1] = pack_bf16x2(y2, y3);
    }
    if (wide) {  // d_out is a multiple of 16
      if (16 * c < left) st_global32(y + 16 * c, w);
    } else {
      if (16 * c < left) *reinterpret_cast<uint4*>(y + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
      if (16 * c + 8 < left) *reinterpret_cast<uint4*>(y + 16 * c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <int kFmt>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMxThreads, 1)
    mx_linear_pair_kernel(const __grid_constant__ MxLinearParams p) {
  constexpr int ST = mx_stages(kFmt), KT = mx_stage_tiles(kFmt);
  constexpr int kSfA = 512 * KT, kSfB = 1024 * KT;  // bytes of a stage's scales
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = sm;
  uint8_t* sB = sA + ST * kMxABytes;
  uint8_t* sSA = sB + ST * kMxBBytes;
  uint8_t* sSB = sSA + ST * kSfA;
  float* sBias = reinterpret_cast<float*>(sSB + ST * kSfB);       // [16 epilogue warps][64]
  // [ST] both CTAs' stage loaded, and the MMAs two stages back complete (rank 0)
  uint64_t* full = reinterpret_cast<uint64_t*>(sBias + 16 * 64);
  uint64_t* empty = full + ST;                                     // [ST] stage consumed
  uint64_t* acc_full = empty + ST;                                 // [2] accumulator complete
  uint64_t* acc_empty = acc_full + 2;                              // [2] accumulator read back (rank 0)
  uint64_t* sh_empty = acc_empty + 2;                              // the shared columns read back (rank 0)
  uint64_t* drain = sh_empty + 1;                                  // MMA abort path
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  __shared__ int abort_flag;

  const int warp = static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int nk = (p.row_bytes + 127) / 128;
  const int pair = static_cast<int>(blockIdx.x >> 1), n_pairs = static_cast<int>(gridDim.x >> 1);
  // units of this pair: pair + i * n_pairs (column tile fastest)
  int n_local = p.units > pair ? (p.units - 1 - pair) / n_pairs + 1 : 0;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 16);  // the epilogue warps of both CTAs that read its own columns
    }
    mbar_init(sh_empty, 16);  // the epilogue warps that read them
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the partner's barriers are initialised before any remote arrival
  tc_fence_after();
  // All 512 columns are allocated, so they begin at address 0: a constant, and
  // with it every TMEM address of the issue loop (read from shared memory,
  // it would pass through a vector register in front of each instruction).
  constexpr uint32_t tbase = 0;
  if (*tmem_slot != tbase) {
    if (threadIdx.x == 0) raise_status(1 << 4);
    n_local = 0;
  }
  // The set-up so far overlaps the end of the kernel in front (a programmatic
  // dependent launch); nothing is read or written before every thread has waited
  // for that kernel. The signal comes after the allocation: a kernel behind that
  // allocates columns can then take none that this one still needs. Layers back to
  // back, without it and with it: mxfp8 4096 x 2304 x 6912 56 -> 52 us,
  // 1024 x 2304 x 2304 18.4 -> 14.8, mxfp4 16 x 2304 x 2304 11.1 -> 10.5.
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ producers (both CTAs)
    // warp 0: elements; warp 3: scales. Each loop runs warp-uniformly and one
    // elected lane issues, so that addresses stay in uniform registers.
    const uint32_t leader = elect_one_sync();
    const bool elements = warp == 0;
    if (leader) {
      tma_prefetch_desc(elements ? &p.x_map : &p.xs_map);
      tma_prefetch_desc(elements ? &p.w_map : &p.ws_map);
    }
    const uint32_t full0 = cluster_addr(full, 0);  // the even CTA's stage barriers
    const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB), sa0 = smem_u32(sSA), sb0 = smem_u32(sSB);
    const uint32_t expect = elements && rank == 0 ? leader : 0u;
    int issued = 0, s = 0;
    uint32_t wrap = 1;  // parity of the last release of stage s (none in the first round)
    bool ok = true;
    for (int i = 0; i < n_local && ok; ++i) {
      const int u = pair + i * n_pairs, piece = u - p.whole;
      const int t = piece < 0 ? u : p.whole + p.piece_tile[piece], nt = t % p.n_tiles;
      const int k0 = piece < 0 ? 0 : p.piece_k0[piece], n = piece < 0 ? nk : p.piece_n[piece];
      // this CTA's rows and columns; rows past the matrix are zero fill and not stored
      const int r0 = (t / p.n_tiles) * 256 + 128 * static_cast<int>(rank);
      const int n0 = nt * kMxTileN, w0 = n0 + 128 * static_cast<int>(rank);
      for (int kc = 0; kc < n; ++kc) {
        if (issued >= ST && !warp_wait_short(&empty[s], wrap, &abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t bar = full0 + static_cast<uint32_t>(s * sizeof(uint64_t));
        if (elements) {
          if (expect) mbar_arrive_expect_tx(&full[s], 2 * mx_stage_bytes(kFmt));
          tma_load_2d_pair_if(leader, a0 + s * kMxABytes, &p.x_map, bar, 128 * (k0 + kc), r0);
          tma_load_2d_pair_if(leader, b0 + s * kMxBBytes, &p.w_map, bar, 128 * (k0 + kc), w0);
        } else {
          tma_load_2d_pair_if(leader, sa0 + s * kSfA, &p.xs_map, bar, 64 * KT * (k0 + kc), r0 >> 7);
          tma_load_2d_pair_if(leader, sb0 + s * kSfB, &p.ws_map, bar, 64 * KT * (k0 + kc), n0 >> 7);
        }
        ++issued;
        if (++s == ST) {
          s = 0;
          wrap ^= 1u;
        }
      }
    }
    if ((!ok || abort_flag) && lane == 0 && rank == 0) {
      // let every copy of the pair land before the CTAs exit (a stage that its
      // second arrival will not reach any more is given the wait's time, 200 ms)
      for (int g = issued - ST < 0 ? 0 : issued - ST; g < issued; ++g) mbar_wait_drain(&full[g % ST], (g / ST) & 1);
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    const uint32_t leader = elect_one_sync();
    // descriptors: constant high words, and low words (the address in 16s,
    // below 2^14 everywhere) that move with the stage
    constexpr uint64_t kMat = 0xFFFFFFFF00000000ull;
    const uint64_t dA = make_sdesc(smem_u32(sA), 16, 1024, kSwizzle128B);
    const uint64_t dB = make_sdesc(smem_u32(sB), 16, 1024, kSwizzle128B);
    const uint64_t dSA = make_sdesc(smem_u32(sSA), 0, 128, kSwizzleNone);
    const uint64_t dSB = make_sdesc(smem_u32(sSB), 0, 128, kSwizzleNone);
    auto at = [&](uint64_t d, uint32_t lo) { return (d & kMat) | lo; };
    const int last_steps = (p.row_bytes - 128 * (nk - 1) + 31) / 32;  // 32-byte steps of the last stage
    int s = 0;
    uint32_t round = 0;
    // the stage's scales: of X, of W; buffers of 48 columns taken in turn
    constexpr uint32_t sfa0 = tbase + 416, sfb0 = sfa0 + 4 * KT;
    uint32_t sfa = sfa0, sfb = sfb0;
    bool ok = true;
    for (int i = 0; i < n_local && ok; ++i) {
      const int a = i & 1;
      if (i >= 2 && !warp_wait(&acc_empty[a], ((i >> 1) - 1) & 1, &abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tacc = tbase + 160 * a;
      const int piece = pair + i * n_pairs - p.whole;
      const int n = piece < 0 ? nk : p.piece_n[piece];
      const int last = piece < 0 || p.piece_k0[piece] + n == nk ? last_steps : 4;
      for (int kc = 0; kc < n; ++kc) {
        if (!warp_wait_short(&full[s], round, &abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t la = static_cast<uint32_t>(dA) + s * (kMxABytes >> 4);
        const uint32_t lb = static_cast<uint32_t>(dB) + s * (kMxBBytes >> 4);
        const uint32_t lsa = static_cast<uint32_t>(dSA) + s * (kSfA >> 4);
        const uint32_t lsb = static_cast<uint32_t>(dSB) + s * (kSfB >> 4);
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          tmem_copy_scales_pair_if(leader, sfa + 4 * j, at(dSA, lsa + 32 * j));
          tmem_copy_scales_pair_if(leader, sfb + 8 * j, at(dSB, lsb + 32 * j));
          tmem_copy_scales_pair_if(leader, sfb + 8 * j + 4, at(dSB, lsb + 32 * (KT + j)));
        }
        auto mma = [&](int steps, uint32_t acc) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            // scale tile and byte of step kk
            constexpr int per = 4 / KT;  // steps that share a tile
            const int j = kk / per, id = kFmt == kMxFp8 ? kk : kFmt == kMxFp4 ? 2 * (kk & 1) : 0;
            umma_pair_mx_if<kFmt>(kk < steps ? leader : 0u, tacc, at(dA, la + 2 * kk), at(dB, lb + 2 * kk),
                                  make_idesc_mx(kFmt, 256, 256, id), sfa + 4 * j, sfb + 8 * j, kk != 0 ? 1u : acc);
          }
        };
        auto shared_read = [&] {  // the last tile's shared columns have been read
          ok = i == 0 || warp_wait_short(sh_empty, (i - 1) & 1, &abort_flag);
          tc_fence_after();
          return ok;
        };
        // The stages between the first and the last of a tile get constants: with
        // one path for all, each MMA's two predicates cost more than they look
        // (nvfp4 51200 x 2304 x 6912 339 us instead of 308, mxfp8 595 instead of 544).
        if (kc == n - 1) {
          if (kc == 0 && !shared_read()) break;
          mma(last, kc != 0 ? 1u : 0u);
        } else if (kc == 0) {
          if (!shared_read()) break;
          mma(4, 0u);
        } else {
          mma(4, 1u);
        }
        // both CTAs' stage may be refilled once these copies and MMAs have read it
        umma_pair_commit_both_if(leader, smem_u32(&empty[s]));
        sfa = 2 * sfa0 + 48 - sfa;
        sfb = 2 * sfb0 + 48 - sfb;
        if (++s == ST) {
          s = 0;
          round ^= 1u;
        }
      }
      if (ok) umma_pair_commit_both_if(leader, smem_u32(&acc_full[a]));
    }
    if (!ok) {
      // wait for every MMA the leader issued before TMEM is released
      umma_pair_commit_if(leader, cluster_addr(drain, 0));
      if (leader) mbar_wait_drain(drain, 0);
      __syncwarp();
    }
  } else if (warp == 2 && rank == 0) {
    // ------------------------------------------------------------ the scale buffers' turns (even CTA)
    int stages = 0;
    for (int i = 0; i < n_local; ++i) {
      const int piece = pair + i * n_pairs - p.whole;
      stages += piece < 0 ? nk : p.piece_n[piece];
    }
    // Stage g may overwrite the scales of stage g - 2. (A slot is not issued again
    // before its arrival here, so its barrier cannot run ahead of this warp.)
    int s = 0, back = ST - 2;
    uint32_t parity = 1;
    for (int g = 0; g < stages; ++g) {
      if (g >= 2 && !warp_wait_short(&empty[back], parity, &abort_flag)) break;
      tc_fence_after();
      tc_fence_before();
      if (lane == 0) mbar_arrive(&full[s]);
      if (++s == ST) s = 0;
      if (++back == ST) {
        back = 0;
        parity ^= 1u;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // warp 4 + 4e + q: TMEM lanes 32q .. 32q + 31, columns 64e .. 64e + 63;
    // each lane stores its row's 128 bytes
    const int q = warp & 3, e = (warp - 4) >> 2;
    const uint32_t lane_addr = tbase + (static_cast<uint32_t>(q * 32) << 16) + 64 * e;
    const uint32_t acce0 = cluster_addr(acc_empty, 0), she0 = cluster_addr(sh_empty, 0);
    float2* bias2 = reinterpret_cast<float2*>(sBias + 64 * (warp - 4));
    const uint32_t bias = smem_u32(bias2);
    auto tile = [&](int i) {  // of unit i (past the last: the first's)
      const int u = i < n_local ? pair + i * n_pairs : pair;
      return u < p.whole ? u : p.whole + p.piece_tile[u - p.whole];
    };
    // the bias of a tile's columns is loaded a tile ahead
    auto load_bias = [&](int i) {
      const int c = tile(i) % p.n_tiles * kMxTileN + 64 * e + 2 * lane;
      if (p.bias == nullptr || c >= p.d_out) return make_float2(0.f, 0.f);  // d_out is a multiple of 8
      return make_float2(__ldcg(p.bias + c), __ldcg(p.bias + c + 1));
    };
    float2 next = load_bias(0);
    for (int i = 0; i < n_local; ++i) {
      const int a = i & 1, t = tile(i), piece = pair + i * n_pairs - p.whole;
      const int nc = (t % p.n_tiles) * kMxTileN + 64 * e;
      const int r = (t / p.n_tiles) * 256 + 128 * static_cast<int>(rank) + 32 * q + lane;
      __syncwarp();  // the last tile's bias has been read
      bias2[lane] = next;
      next = load_bias(i + 1);
      const bool sh = (e >> 1) == (a ^ 1);  // these warps' columns reach into the shared ones
      if (!warp_wait_short(&acc_full[a], (i >> 1) & 1, &abort_flag)) break;
      tc_fence_after();
      uint32_t v[64];
      tmem_ld32(lane_addr + 160 * a, v);
      tmem_ld32(lane_addr + 160 * a + 32, v + 32);
      tmem_ld_wait32(v);
      tmem_ld_wait32(v + 32);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(sh ? she0 : acce0 + static_cast<uint32_t>(a * sizeof(uint64_t)));
      if (piece >= 0) {
        float* part = p.part + (static_cast<size_t>(piece) * 256 + 128 * rank + 32 * q + lane) * 256 + 64 * e;
        if (r < p.M) {
#pragma unroll
          for (int c = 0; c < 8; ++c) st_global32(part + 8 * c, v + 8 * c);
        }
      } else if (r < p.M) {
        __nv_bfloat16* y = p.Y + static_cast<size_t>(r) * p.d_out + nc;
        if (p.act == 1) mx_store_row<true>(v, p.alpha, bias, y, p.d_out - nc, p.wide);
        else mx_store_row<false>(v, p.alpha, bias, y, p.d_out - nc, p.wide);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the partner's MMAs, copies and arrivals are done
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(*tmem_slot, 512);
}

// The tiles that were split: act(alpha sum of the pieces + bias), the pieces added
// in order. A thread takes 8 columns of a row.
struct MxMergeParams {
  const float* part;
  const float* bias;
  __nv_bfloat16* Y;
  float alpha;
  int M, d_out, act, n_tiles, whole, split;
};
__global__ void __launch_bounds__(256) mx_linear_merge_kernel(const MxMergeParams p) {
  // the pieces are stored; no load here is of the read-only kind, which the
  // compiler may move up past the wait
  pdl_wait();
  const int tile = blockIdx.x >> 5, t = p.whole + tile;  // 32 CTAs of 8 rows for a tile
  const int row = (blockIdx.x & 31) * 8 + (threadIdx.x >> 5), col = (threadIdx.x & 31) * 8;
  const int r = (t / p.n_tiles) * 256 + row, c = (t % p.n_tiles) * kMxTileN + col;
  if (r >= p.M || c >= p.d_out) return;  // d_out is a multiple of 8
  const float* part = p.part + (static_cast<size_t>(tile) * p.split * 256 + row) * 256 + col;
  float f[8] = {};
  for (int k = 0; k < p.split; ++k) {
    const float4 a = __ldcg(reinterpret_cast<const float4*>(part + static_cast<size_t>(k) * 65536));
    const float4 b = __ldcg(reinterpret_cast<const float4*>(part + static_cast<size_t>(k) * 65536) + 1);
    f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
    f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = fmaf(f[k], p.alpha, p.bias != nullptr ? __ldcg(p.bias + c + k) : 0.f);
  if (p.act == 1) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) f2_unpack(gelu_tanh_2(f2_pack(f[k], f[k + 1])), f[k], f[k + 1]);
  }
  store8(p.Y + static_cast<size_t>(r) * p.d_out + c, f);
}

}  // namespace safe
