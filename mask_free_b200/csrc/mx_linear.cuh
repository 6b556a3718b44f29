// mx_linear.cuh - row-wise layers of the row-selective block with microscaled operands.
//
//     Y[r, :] = act( alpha * sum_c X[r, c] W[:, c] + bias )
// X and W are microscaled matrices (mx_quant.cuh) of the same format; the
// tensor core multiplies the 8- or 4-bit elements, applies both block scales
// to each block's products and adds in fp32 (tcgen05.mma .block_scale).
//
// linear_pair_kernel's structure with other operands: a CTA pair computes
// 256 x 192 output tiles, each CTA 128 rows. A stage of the ring is 128
// bytes of every row (128 e4m3 or 256 e2m1 elements, four MMA steps of 32
// bytes) with the scales that belong to them:
//   A       the CTA's 128 rows x 128 B            16 KB
//   B       the CTA's 96 of the 192 W rows        12 KB
//   scale A of the CTA's own rows (one scale tile for each 4 scales of a row)
//   scale B of all 192 W rows, in both CTAs: two scale tiles high, since a
//           tile of columns begins in the middle of one when its index is odd
// Scales travel shared memory -> TMEM by tcgen05.cp (32 lanes x 16 B, copied
// to all four lane quarters) right before the MMAs that use them; copies and
// MMAs of one thread run in order, and two scale buffers let the next
// stage's copies pass the current MMAs. TMEM: two 192-column accumulators
// (tile i uses i & 1) and the two scale buffers of 48 columns: 480 of 512.
// With 256 columns the second accumulator would not fit beside the scales,
// and every tile's MMAs would wait for the last tile's epilogue.
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

struct MxLinearParams {
  CUtensorMap x_map;   // bytes [M, row bytes], box 128 x 128, 128B swizzle
  CUtensorMap w_map;   // bytes [d_out, row bytes], box 128 x 96, 128B swizzle
  CUtensorMap xs_map;  // scale tiles as 8-byte words [row blocks, tiles * 64], box (tiles of a stage * 64) x 1
  CUtensorMap ws_map;  // the same of W, box (tiles of a stage * 64) x 2
  const float* bias;   // [d_out] or null
  __nv_bfloat16* Y;    // [M, d_out]
  float alpha;
  int M, row_bytes, d_out, act;
  int n_tiles, tiles;  // column tiles (192), all tiles
};

constexpr int kMxTileN = 192;
constexpr int kMxStages = 6;
constexpr int kMxABytes = 128 * 128;
constexpr int kMxBBytes = 96 * 128;
// scale tiles along a row in a stage: 128 B hold 4 (mxfp8), 8 (mxfp4) or 16 (nvfp4) scales
__host__ __device__ constexpr int mx_stage_tiles(int fmt) { return fmt == kMxFp8 ? 1 : fmt == kMxFp4 ? 2 : 4; }
__host__ __device__ constexpr int mx_stage_bytes(int fmt) { return kMxABytes + kMxBBytes + 3 * 512 * mx_stage_tiles(fmt); }
__host__ __device__ constexpr int mx_linear_smem(int fmt) { return 1024 + kMxStages * mx_stage_bytes(fmt) + 256; }

template <int kFmt>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLinThreads, 1)
    mx_linear_pair_kernel(const __grid_constant__ MxLinearParams p) {
  constexpr int ST = kMxStages, KT = mx_stage_tiles(kFmt);
  constexpr int kSfA = 512 * KT, kSfB = 1024 * KT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = sm;
  uint8_t* sB = sA + ST * kMxABytes;
  uint8_t* sSA = sB + ST * kMxBBytes;
  uint8_t* sSB = sSA + ST * kSfA;
  uint64_t* full = reinterpret_cast<uint64_t*>(sSB + ST * kSfB);  // [ST] both CTAs' stage loaded (rank 0)
  uint64_t* empty = full + ST;                                     // [ST] stage consumed
  uint64_t* acc_full = empty + ST;                                 // [2] accumulator complete
  uint64_t* acc_empty = acc_full + 2;                              // [2] accumulator read back (rank 0)
  uint64_t* drain = acc_empty + 2;                                 // MMA abort path
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int nk = (p.row_bytes + 127) / 128;
  const int pair = static_cast<int>(blockIdx.x >> 1), n_pairs = static_cast<int>(gridDim.x >> 1);
  // 256 x 192 tiles of this pair: t = pair + i * n_pairs (column tile fastest)
  const int n_local = p.tiles > pair ? (p.tiles - 1 - pair) / n_pairs + 1 : 0;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 512);  // every epilogue thread of both CTAs
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the partner's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      tma_prefetch_desc(&p.x_map);
      tma_prefetch_desc(&p.w_map);
      tma_prefetch_desc(&p.xs_map);
      tma_prefetch_desc(&p.ws_map);
    }
    const uint32_t full0 = cluster_addr(full, 0);  // the even CTA's stage barriers
    int issued = 0;
    bool ok = true;
    for (int i = 0; i < n_local && ok; ++i) {
      const int t = pair + i * n_pairs, nt = t % p.n_tiles;
      // this CTA's rows and columns; rows past the matrix are zero fill and not stored
      const int r0 = (t / p.n_tiles) * 256 + 128 * static_cast<int>(rank);
      const int n0 = nt * kMxTileN, nb = n0 + 96 * static_cast<int>(rank);
      for (int kc = 0; kc < nk; ++kc) {
        const int g = i * nk + kc, s = g % ST;
        if (g >= ST && !warp_wait(&empty[s], ((g / ST) - 1) & 1, &abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * mx_stage_bytes(kFmt));
          const uint32_t bar = full0 + static_cast<uint32_t>(s * sizeof(uint64_t));
          tma_load_2d_pair(sA + s * kMxABytes, &p.x_map, bar, 128 * kc, r0);
          tma_load_2d_pair(sB + s * kMxBBytes, &p.w_map, bar, 128 * kc, nb);
          tma_load_2d_pair(sSA + s * kSfA, &p.xs_map, bar, 64 * KT * kc, r0 >> 7);
          tma_load_2d_pair(sSB + s * kSfB, &p.ws_map, bar, 64 * KT * kc, n0 >> 7);
        }
        __syncwarp();
        issued = g + 1;
      }
    }
    if ((!ok || abort_flag) && lane == 0 && rank == 0) {
      // let every copy of the pair land before the CTAs exit
      for (int g = issued - ST < 0 ? 0 : issued - ST; g < issued; ++g) mbar_wait_drain(&full[g % ST], (g / ST) & 1);
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    const uint32_t leader = elect_one_sync();
    const uint32_t empty0 = cluster_addr(empty, 0), empty1 = cluster_addr(empty, 1);
    const uint32_t accf0 = cluster_addr(acc_full, 0), accf1 = cluster_addr(acc_full, 1);
    const int last_steps = (p.row_bytes - 128 * (nk - 1) + 31) / 32;  // 32-byte steps of the last stage
    bool ok = true;
    for (int i = 0; i < n_local && ok; ++i) {
      const int a = i & 1;
      if (i >= 2 && !warp_wait(&acc_empty[a], ((i >> 1) - 1) & 1, &abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tacc = tbase + kMxTileN * a;
      // an odd column tile begins 64 rows (two TMEM columns) into its first scale tile
      const uint32_t sfb_shift = ((pair + i * n_pairs) % p.n_tiles) & 1 ? 2u : 0u;
      for (int kc = 0; kc < nk; ++kc) {
        const int g = i * nk + kc, s = g % ST;
        if (!warp_wait(&full[s], (g / ST) & 1, &abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a0 = smem_u32(sA + s * kMxABytes), b0 = smem_u32(sB + s * kMxBBytes);
        const uint32_t sa0 = smem_u32(sSA + s * kSfA), sb0 = smem_u32(sSB + s * kSfB);
        const uint32_t sfa = tbase + 2 * kMxTileN + 48u * (g & 1), sfb = sfa + 16;
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          tmem_copy_scales_pair_if(leader, sfa + 4 * j, make_sdesc(sa0 + 512 * j, 0, 128, kSwizzleNone));
          tmem_copy_scales_pair_if(leader, sfb + 8 * j, make_sdesc(sb0 + 512 * j, 0, 128, kSwizzleNone));
          tmem_copy_scales_pair_if(leader, sfb + 8 * j + 4, make_sdesc(sb0 + 512 * (KT + j), 0, 128, kSwizzleNone));
        }
        const int steps = kc == nk - 1 ? last_steps : 4;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          // scale tile and byte of step kk
          constexpr int per = 4 / KT;  // steps that share a tile
          const int j = kk / per, id = kFmt == kMxFp8 ? kk : kFmt == kMxFp4 ? 2 * (kk & 1) : 0;
          if (kk < steps)
            umma_pair_mx_if<kFmt>(leader, tacc, make_sdesc(a0 + 32 * kk, 16, 1024, kSwizzle128B),
                                  make_sdesc(b0 + 32 * kk, 16, 1024, kSwizzle128B),
                                  make_idesc_mx(kFmt, 256, kMxTileN, id), sfa + 4 * j, sfb + 8 * j + sfb_shift,
                                  (kc | kk) != 0 ? 1u : 0u);
        }
        // both CTAs' stage may be refilled once these copies and MMAs have read it
        const uint32_t so = static_cast<uint32_t>(s * sizeof(uint64_t));
        umma_pair_commit_if(leader, empty0 + so);
        umma_pair_commit_if(leader, empty1 + so);
      }
      if (ok) {
        const uint32_t ao = static_cast<uint32_t>(a * sizeof(uint64_t));
        umma_pair_commit_if(leader, accf0 + ao);
        umma_pair_commit_if(leader, accf1 + ao);
      }
    }
    if (!ok) {
      // wait for every MMA the leader issued before TMEM is released
      umma_pair_commit_if(leader, cluster_addr(drain, 0));
      if (leader) mbar_wait_drain(drain, 0);
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // warp 4 + 4e + q: TMEM lanes 32q .. 32q + 31, columns 96e .. 96e + 95
    const int q = warp & 3, row = q * 32 + lane, e = (warp - 4) >> 2;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t acce0 = cluster_addr(acc_empty, 0);
    for (int i = 0; i < n_local; ++i) {
      const int a = i & 1;
      if (!warp_wait(&acc_full[a], (i >> 1) & 1, &abort_flag)) break;
      tc_fence_after();
      const int t = pair + i * n_pairs, n0 = (t % p.n_tiles) * kMxTileN;
      const int r = (t / p.n_tiles) * 256 + 128 * static_cast<int>(rank) + row;
      const bool valid = r < p.M;
      __nv_bfloat16* yrow = p.Y + static_cast<size_t>(valid ? r : 0) * p.d_out;
#pragma unroll 1
      for (int c = 3 * e; c < 3 * e + 3; ++c) {
        uint32_t v[32];
        tmem_ld32(tbase + lane_addr + kMxTileN * a + 32 * c, v);
        tmem_ld_wait32(v);
        if (c == 3 * e + 2) {
          // the accumulator is released to the even CTA's issuer
          tc_fence_before();
          mbar_arrive_cluster(acce0 + static_cast<uint32_t>(a * sizeof(uint64_t)));
        }
        const int nc = n0 + 32 * c;
        if (nc >= p.d_out) continue;
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float f0 = __uint_as_float(v[2 * k]) * p.alpha, f1 = __uint_as_float(v[2 * k + 1]) * p.alpha;
          if (p.bias != nullptr && nc + 2 * k < p.d_out) {  // d_out is even
            f0 += __ldg(p.bias + nc + 2 * k);
            f1 += __ldg(p.bias + nc + 2 * k + 1);
          }
          if (p.act == 1) {
            f0 = gelu_tanh_f(f0);
            f1 = gelu_tanh_f(f1);
          }
          pk[k] = pack_bf16x2(f0, f1);
        }
        if (valid) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (nc + 8 * u < p.d_out)
              *reinterpret_cast<uint4*>(yrow + nc + 8 * u) =
                  make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the partner's MMAs, copies and arrivals are done
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tbase, 512);
}

}  // namespace safe
