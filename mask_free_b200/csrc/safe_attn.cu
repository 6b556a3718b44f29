// safe_attn.cu - host side of the C ABI declared in include/safe_attn.h.
//
// One translation unit: it includes every kernel of the library, validates
// arguments on the host, encodes the TMA tensor maps and launches on the
// caller's stream. The library allocates no device memory.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "safe_attn.h"
#include "sm100.cuh"
#include "flash_attn.cuh"
#include "cross_attn.cuh"
#include "aux_kernels.cuh"
#include "guidance.cuh"
#include "linear.cuh"
#include "mx_quant.cuh"
#include "norm.cuh"
#include "rope.cuh"
#include "mx_linear.cuh"

using namespace safe;

namespace {

constexpr int kAbiVersion = 7;
constexpr float kLog2e = 1.4426950408889634f;

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool supported_d(int d) { return d == 64 || d == 96 || d == 128; }

// The attention kernels take each row's maximum of the unscaled logits and
// scale it afterwards, which is the row's largest scaled logit only for a
// positive scale; padding keys are masked with -inf before scaling.
bool scale_ok(float scale) { return std::isfinite(scale) && scale > 0.f; }

safe_status launch_status() {
  return cudaGetLastError() == cudaSuccess ? SAFE_OK : SAFE_ERR_CUDA;
}

// ---------------------------------------------------------------- TMA maps
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

int chunk_width(int d, int c) { return (d - 64 * c) >= 64 ? 64 : (d - 64 * c); }

CUtensorMapSwizzle chunk_swizzle(int d, int c) {
  return chunk_width(d, c) == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
}

// [B, rows, H, d] bf16 tensor viewed as 4-D (d, H, rows, B); box = one
// chunk of the head dim x 1 head x 128 rows x 1 sample. Rows past `rows`
// read as zero.
bool encode_rows_map(CUtensorMap* map, const void* base, int B, int rows, int H, int d, int c) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(H) * d * 2,
                           static_cast<cuuint64_t>(rows) * H * d * 2};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(chunk_width(d, c)), 1, 128, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, chunk_swizzle(d, c), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Same 4-D view with the equal-width V chunks of the flash kernel (32 wide
// with the 64B swizzle for d = 96, else 64 wide with the 128B swizzle).
bool encode_v_map(CUtensorMap* map, const void* base, int B, int rows, int H, int d) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const int w = d == 96 ? 32 : 64;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(H) * d * 2,
                           static_cast<cuuint64_t>(rows) * H * d * 2};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(w), 1, 128, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, w == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [B*N, H*d] 2-D view for tile::gather4 (box one row high).
// 2-D bf16 matrix [outer, inner] (row pitch = inner), 128B swizzle; box
// box_inner x box_outer (the row-wise layers' X, box 64 x 1 for gather4, and
// W^T, box 64 x 256).
bool encode_matrix_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint32_t box_inner,
                       uint32_t box_outer) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * 2};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t es[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_gather_map(CUtensorMap* map, const void* base, int B, int N, int H, int d, int c) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(H) * d, static_cast<cuuint64_t>(B) * N};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(H) * d * 2};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(chunk_width(d, c)), 1};
  cuuint32_t es[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, chunk_swizzle(d, c), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int nchunks(int d) { return (d + 63) / 64; }

// ---------------------------------------------------------------- launches
int device_sms() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess) return sms;
  static int cached[64] = {};
  if (dev >= 0 && dev < 64 && cached[dev] > 0) return cached[dev];
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (dev >= 0 && dev < 64) cached[dev] = sms;
  return sms;
}

// How the (b, h, 256-row block) work units of one flash launch are spread
// over the SMs: `full` whole units first, then the remaining units split
// into `split` key ranges each (see FlashParams).
struct FlashPlan {
  int units, full, split, tail;
  size_t ws_o, ws_ml, ws_bytes;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

FlashPlan plan_flash(int B, int H, int n_q, int N, int d, int sms) {
  FlashPlan pl{};
  const int n_mblk = (n_q + 255) / 256;
  const int n_kv = (N + 127) / 128;
  pl.units = n_mblk * H * B;
  pl.full = pl.units;
  pl.split = 1;
  pl.tail = 0;
  // Cost model in key-tile steps (calibrated on B200): a whole unit costs
  // n_kv + 2, a part n_kv / s + 8 (set-up, pipeline fill and drain, partial
  // store, and the spread of finish times across SMs), the merge launch
  // about 3. Only the last waves are split; each part keeps at least 4 key
  // tiles.
  const double whole = n_kv + 2.0;
  double best = static_cast<double>((pl.units + sms - 1) / sms) * whole;
  const int max_split = n_kv / 4 < kMaxSplit ? n_kv / 4 : kMaxSplit;  // the merge kernel takes at most kMaxSplit parts
  for (int fw = pl.units / sms; fw >= 0 && fw >= pl.units / sms - 1; --fw) {
    const int f = fw * sms, r = pl.units - f;
    if (r <= 0) continue;
    for (int sp = 2; sp <= max_split; ++sp) {
      const double rounds = static_cast<double>((static_cast<long long>(r) * sp + sms - 1) / sms);
      const double cost = fw * whole + rounds * (static_cast<double>(n_kv) / sp + 8.0) + 3.0;
      if (cost < 0.99 * best) {
        best = cost;
        pl.full = f;
        pl.split = sp;
        pl.tail = r;
      }
    }
  }
  if (pl.split > 1) {
    const size_t slots = static_cast<size_t>(pl.tail) * pl.split * 256;
    pl.ws_o = 0;  // bf16 O / l of the parts
    pl.ws_ml = align256(slots * d * 2);
    pl.ws_bytes = pl.ws_ml + align256(slots * sizeof(float2));
  }
  return pl;
}

template <int D, bool kAsm>
safe_status launch_flash(FlashParams& p, void* ws, size_t ws_bytes, cudaStream_t s) {
  constexpr int smem = flash_smem_bytes<D>();
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(flash_fwd_kernel<D, kAsm>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr_err != cudaSuccess) return SAFE_ERR_CUDA;
  FlashPlan pl = plan_flash(p.B, p.H, p.n_q, p.N, D, device_sms());
  if (pl.split > kMaxSplit) return SAFE_ERR_UNSUPPORTED;  // the merge takes at most kMaxSplit parts
  if (pl.split > 1 && (!aligned16(ws) || ws_bytes < pl.ws_bytes)) {
    pl.full = pl.units;  // no workspace: whole units only
    pl.split = 1;
    pl.tail = 0;
  }
  p.n_mblk = (p.n_q + 255) / 256;
  p.full_units = pl.full;
  p.split = pl.split;
  p.ws_ob = nullptr;
  p.ws_ml = nullptr;
  if (pl.split > 1) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    p.ws_ob = reinterpret_cast<__nv_bfloat16*>(w + pl.ws_o);
    p.ws_ml = reinterpret_cast<float2*>(w + pl.ws_ml);
    for (int c = 0; c < nchunks(D); ++c)
      if (!encode_rows_map(&p.ws_map[c], p.ws_ob, 1, pl.tail * pl.split * 256, 1, D, c)) return SAFE_ERR_CUDA;
  }
  const unsigned grid = static_cast<unsigned>(pl.full + pl.tail * pl.split);
  // both launches are programmatic dependents of what precedes them in the
  // stream: their set-up overlaps its tail, and each waits (griddepcontrol)
  // for it before reading anything
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFlashThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, flash_fwd_kernel<D, kAsm>, p) != cudaSuccess) return SAFE_ERR_CUDA;
  if (pl.split > 1) {
    cfg.gridDim = dim3((pl.tail * 256 + 7) / 8);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, flash_merge_kernel<D>, p, pl.tail) != cudaSuccess) return SAFE_ERR_CUDA;
  }
  return launch_status();
}

// assembled: SRSU with the keys of S taken from p.k_cur / p.v_cur
safe_status dispatch_flash(int d, FlashParams& p, void* ws, size_t ws_bytes, cudaStream_t s, bool assembled = false) {
  switch (d) {
    case 64: return assembled ? launch_flash<64, true>(p, ws, ws_bytes, s) : launch_flash<64, false>(p, ws, ws_bytes, s);
    case 96: return assembled ? launch_flash<96, true>(p, ws, ws_bytes, s) : launch_flash<96, false>(p, ws, ws_bytes, s);
    case 128:
      return assembled ? launch_flash<128, true>(p, ws, ws_bytes, s) : launch_flash<128, false>(p, ws, ws_bytes, s);
    default: return SAFE_ERR_UNSUPPORTED;
  }
}

template <int D, bool kSep, bool kO>
cudaError_t cross_smem_attr() {
  return cudaFuncSetAttribute(cross_attn_kernel<D, kSep, kO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kCrossMaxSmem);
}

template <int D>
safe_status launch_cross(CrossParams& p, cudaStream_t s) {
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cross_smem_attr<D, false, true>();
    if (attr_err == cudaSuccess) attr_err = cross_smem_attr<D, false, false>();
    if constexpr (D <= 96) {
      if (attr_err == cudaSuccess) attr_err = cross_smem_attr<D, true, true>();
      if (attr_err == cudaSuccess) attr_err = cross_smem_attr<D, true, false>();
    }
  });
  if (attr_err != cudaSuccess) return SAFE_ERR_CUDA;
  // one CTA per SM (each holds all of TMEM), a few per (b, h), each streaming
  // a contiguous range of query tiles
  const int n_tiles = (p.nq + 127) / 128;
  int per_bh = device_sms() / (p.B * p.H);
  per_bh = per_bh < 1 ? 1 : (per_bh > n_tiles ? n_tiles : per_bh);
  p.qs = cross_slots<D>(p.M);
  dim3 grid(per_bh, p.H, p.B);
  const int smem = cross_smem_bytes<D>(p.M);
  const bool o = p.O != nullptr;  // else PCSP partials only
  bool sep = false;
  if constexpr (D <= 96) sep = cross_sep_p<D>(p.M);
  if constexpr (D <= 96) {
    if (sep) {
      if (o)
        cross_attn_kernel<D, true, true><<<grid, kCrossThreads, smem, s>>>(p);
      else
        cross_attn_kernel<D, true, false><<<grid, kCrossThreads, smem, s>>>(p);
    }
  }
  if (!sep) {
    if (o)
      cross_attn_kernel<D, false, true><<<grid, kCrossThreads, smem, s>>>(p);
    else
      cross_attn_kernel<D, false, false><<<grid, kCrossThreads, smem, s>>>(p);
  }
  return launch_status();
}

safe_status dispatch_cross(int d, CrossParams& p, cudaStream_t s) {
  switch (d) {
    case 64: return launch_cross<64>(p, s);
    case 96: return launch_cross<96>(p, s);
    case 128: return launch_cross<128>(p, s);
    default: return SAFE_ERR_UNSUPPORTED;
  }
}

bool sizes_ok(int B, int N, int H) {
  return B >= 1 && N >= 1 && H >= 1 && B <= 65535 && H <= 65535 &&
         static_cast<int64_t>(B) * N <= INT_MAX;
}

// Fill the query maps of a cross-attention launch (dense or gathered rows).
safe_status fill_cross(CrossParams& p, const void* Q, const int32_t* q_idx, int nq, const void* Ky, const void* Vy,
                       const int32_t* valid_len, const float* w, void* O, float* partial, int B, int N, int M, int H,
                       int d, float scale) {
  p = CrossParams{};
  for (int c = 0; c < nchunks(d); ++c) {
    if (q_idx == nullptr) {
      if (!encode_rows_map(&p.q_map[c], Q, B, N, H, d, c)) return SAFE_ERR_CUDA;
    } else {
      if (!encode_gather_map(&p.qg_map[c], Q, B, N, H, d, c)) return SAFE_ERR_CUDA;
    }
  }
  if (O != nullptr)
    for (int c = 0; c < nchunks(d); ++c)
      if (!encode_rows_map(&p.o_map[c], O, B, nq, H, d, c)) return SAFE_ERR_CUDA;
  p.Ky = static_cast<const __nv_bfloat16*>(Ky);
  p.Vy = static_cast<const __nv_bfloat16*>(Vy);
  p.valid_len = valid_len;
  p.q_idx = q_idx;
  p.w = w;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.partial = partial;
  p.B = B;
  p.N = N;
  p.M = M;
  p.H = H;
  p.nq = nq;
  p.scale_log2 = scale * kLog2e;
  p.gather = q_idx != nullptr;
  return SAFE_OK;
}

}  // namespace

// ---------------------------------------------------------------- allocation-free PCSP
// Scratch for safe_pcsp_topk_noalloc: the per-head partial scores [B, H, N]
// live in this fixed array, which every GPU that loads the library keeps
// until the process exits. Host code must not use the name as an address (it
// is only a host-side stand-in); the device address comes from
// cudaGetSymbolAddress, looked up once per device below.
constexpr size_t kNoAllocScratchFloats = size_t(1) << 21;  // 2 Mi floats = 8 MiB
static __device__ __align__(256) float g_pcsp_noalloc_scratch[kNoAllocScratchFloats];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_noalloc_mu;
void* g_noalloc_ptr[kMaxDevices] = {};

// Device address of the scratch array on the current device (set up on the
// first call made with that device current).
safe_status noalloc_scratch(void** out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return SAFE_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return SAFE_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_pcsp_noalloc_scratch) != cudaSuccess || p == nullptr) return SAFE_ERR_CUDA;
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return SAFE_OK;
}

// Parameters of an SRSU launch (tensor maps of Q or its gather map and of the
// cache K / V); false when a map cannot be encoded.
bool fill_srsu(FlashParams& p, const void* Q, int q_compact, const int32_t* S, int k, const void* Kc, const void* Vc,
               void* O_S, float* lse, int B, int N, int H, int d, float scale) {
  if (!encode_v_map(&p.v_map, Vc, B, N, H, d)) return false;
  for (int c = 0; c < nchunks(d); ++c) {
    bool ok = encode_rows_map(&p.k_map[c], Kc, B, N, H, d, c);
    ok = ok && (q_compact ? encode_rows_map(&p.q_map[c], Q, B, k, H, d, c)
                          : encode_gather_map(&p.qg_map[c], Q, B, N, H, d, c));
    ok = ok && encode_rows_map(&p.o_map[c], O_S, B, k, H, d, c);
    if (!ok) return false;
  }
  p.S = S;
  p.O = static_cast<__nv_bfloat16*>(O_S);
  p.lse = lse;
  p.B = B;
  p.N = N;
  p.H = H;
  p.n_q = k;
  p.scale_log2 = scale * kLog2e;
  p.gather = q_compact ? 0 : 1;
  return true;
}

// With the query rows gathered from a full-size Q and room for them in the
// workspace (safe_srsu_workspace_bytes): copy the rows of S into the end of
// the workspace as a compact [B, k, H, d] tensor and point Q there, so the
// kernel loads each query tile by one tiled copy instead of per-row gathers;
// the rest of the workspace is left for the key split. False on a launch
// error.
bool srsu_compact_q(const void*& Q, int& q_compact, const int32_t* S, int k, int B, int N, int H, int d, void* ws,
                    size_t& ws_bytes, cudaStream_t s) {
  if (q_compact || ws == nullptr || !aligned16(ws)) return true;
  const size_t split = align256(safe_attn_workspace_bytes(B, k, N, H, d));
  const size_t need = split + static_cast<size_t>(B) * k * H * d * 2;
  if (ws_bytes < need) return true;
  const long long rows = static_cast<long long>(B) * k;
  if ((rows + 7) / 8 > INT_MAX) return true;
  void* qc = static_cast<uint8_t*>(ws) + split;
  gather_rows_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, s>>>(static_cast<const uint4*>(Q), S,
                                                                           static_cast<uint4*>(qc), B, N, k,
                                                                           H * d / 8);
  if (cudaGetLastError() != cudaSuccess) return false;
  Q = qc;
  q_compact = 1;
  ws_bytes = split;
  return true;
}

// ---------------------------------------------------------------- norm, positions, microscaled layers
// Bytes of a floating type, 0 for the others.
size_t float_size(int dtype) {
  return dtype == SAFE_F32 ? 4 : dtype == SAFE_F16 || dtype == SAFE_BF16 ? 2 : 0;
}
bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// Whether two ranges of memory share a byte (a null one shares none).
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && an > 0 && bn > 0 && x < y + bn && y < x + an;
}
// A strided [B, R, H, d] tensor (strides in elements, the head dim contiguous).
struct View4 {
  uintptr_t at;
  int64_t size[3], stride[3];  // sample, row, head
  int d;
};
// Whether blocks of `block` elements at the given strides share no element; dims
// of one entry do not count. Covers the layouts in which each dim's stride
// passes over all of the dims inside it.
bool nested(int64_t block, const int64_t* size, const int64_t* stride, int n) {
  bool used[3] = {};
  for (int i = 0; i < n; ++i) {
    int m = -1;
    for (int j = 0; j < n; ++j)
      if (!used[j] && size[j] > 1 && (m < 0 || stride[j] < stride[m])) m = j;
    if (m < 0) return true;
    if (stride[m] < block) return false;
    block += (size[m] - 1) * stride[m];
    used[m] = true;
  }
  return true;
}
int64_t extent(const View4& t, bool samples, bool rows) {
  return t.d + (t.size[2] - 1) * t.stride[2] + (rows ? (t.size[1] - 1) * t.stride[1] : 0) +
         (samples ? (t.size[0] - 1) * t.stride[0] : 0);
}
// Whether two views of the same samples and rows share no element: apart as a
// whole, or side by side in each row or in each sample (views of one fused tensor).
bool apart(const View4& s, const View4& t, size_t e) {
  const View4 &a = s.at <= t.at ? s : t, &b = s.at <= t.at ? t : s;
  const uintptr_t gap = b.at - a.at;
  if (gap >= static_cast<uintptr_t>(extent(a, true, true)) * e) return true;
  if (gap % e != 0 || a.size[0] != b.size[0] || a.size[1] != b.size[1]) return false;
  const int64_t off = static_cast<int64_t>(gap / e);
  for (int outer = 2; outer >= 1; --outer) {  // side by side in a row, in a sample
    const bool rows = outer == 1;
    bool same = true;
    for (int i = 0; i < outer; ++i) same = same && (a.size[i] == 1 || a.stride[i] == b.stride[i]);
    if (same && off >= extent(a, false, rows) && nested(off + extent(b, false, rows), a.size, a.stride, outer)) return true;
  }
  return false;
}
constexpr int kMxMaxD = 1 << 20;  // keeps the positions of 128 rows below 2^31
constexpr int64_t kMxMaxRows = INT_MAX - 255;  // and the rows of the last, partial tile
int mx_block(int fmt) { return fmt == SAFE_NVFP4 ? 16 : 32; }
// Scale tiles along a row of D elements.
int mx_tiles(int D, int fmt) { return (D / mx_block(fmt) + 3) / 4; }
// The tensor's factor: 1 for the formats that have none; for nvfp4 within a
// range that keeps 6 g, its inverse and every product with it normal numbers.
bool mx_factor_ok(int fmt, float g) {
  if (fmt < SAFE_MXFP8 || fmt > SAFE_NVFP4 || !std::isfinite(g)) return false;
  return fmt == SAFE_NVFP4 ? g >= 0x1p-100f && g <= 0x1p100f : g == 1.f;
}

// Sets a kernel's shared-memory limit once for each device. (The kernel is a
// template argument: instances of one kernel template share their type.)
template <auto kKernel>
bool allow_smem(int bytes) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < 64 && done[dev]) return true;
  if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64) done[dev] = true;
  return true;
}

FastDiv fast_div(uint32_t d) {  // d >= 2
  uint32_t l = 1;
  while ((1ull << l) < d) ++l;
  return FastDiv{static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), l - 1};
}

constexpr int kNormMaxVec = 512 * 8 * 10;  // longest row that rms_norm_kernel holds in registers

// Behind norm_order_kernel the norm is its programmatic dependent.
template <typename K>
safe_status norm_launch(K kernel, int64_t ctas, int threads, const NormParams& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = p.mark != nullptr ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return SAFE_ERR_CUDA;
  return launch_status();
}

template <typename T, int kMode, int NV, int TPR>
safe_status norm_launch(const NormParams& p, cudaStream_t s) {
  constexpr int rows_cta = TPR <= 32 ? 128 / TPR : 1;
  return norm_launch(rms_norm_kernel<T, kMode, NV, TPR>, (p.rows_pad + rows_cta - 1) / rows_cta, TPR <= 32 ? 128 : TPR, p, s);
}

// The fewest threads that hold a row in a few units each: part of a warp for
// short rows (51200 rows of 128: 14 us, with a warp for each 25), a warp, 96 or 128 threads,
// 512.
template <typename T, int kMode>
safe_status launch_norm_units(const NormParams& p, int units, cudaStream_t s) {
  if (kMode == kNormVec && units <= 8 && p.q == nullptr) return norm_launch<T, kNormVec, 2, 4>(p, s);
  if (units <= 32) return norm_launch<T, kMode, 2, 16>(p, s);
  if (units <= 64) return norm_launch<T, kMode, 2, 32>(p, s);
  if (units <= 128) return norm_launch<T, kMode, 4, 32>(p, s);
  if (units <= 192) return norm_launch<T, kMode, 2, 96>(p, s);
  if (units <= 256) return norm_launch<T, kMode, 2, 128>(p, s);
  if (units <= 288) return norm_launch<T, kMode, 3, 96>(p, s);
  if (units <= 384) return norm_launch<T, kMode, 3, 128>(p, s);
  if (units <= 512) return norm_launch<T, kMode, 4, 128>(p, s);
  if (units <= 896) return norm_launch<T, kMode, 7, 128>(p, s);
  if (units <= 1280) return norm_launch<T, kMode, 10, 128>(p, s);
  if (kMode == kNormShift || units <= 2560) return norm_launch<T, kMode, 5, 512>(p, s);
  return norm_launch<T, kNormVec, 10, 512>(p, s);
}

template <typename T>
safe_status launch_norm(const NormParams& p, int mode, cudaStream_t s) {
  if (mode == kNormVec && p.D <= kNormMaxVec) return launch_norm_units<T, kNormVec>(p, p.D / 8, s);
  if (mode == kNormShift && p.D > 64 && p.D <= 20480 - 14) return launch_norm_units<T, kNormShift>(p, (p.D + 14) / 8, s);
  if (p.D <= 8) return norm_launch<T, kNormOne, 2, 4>(p, s);
  if (p.D <= 64) return norm_launch<T, kNormOne, 4, 16>(p, s);
  if (p.D <= 32 * 10) return norm_launch<T, kNormOne, 10, 32>(p, s);
  if (p.D <= 128 * 10) return norm_launch<T, kNormOne, 10, 128>(p, s);
  if (p.D <= 128 * 20) return norm_launch<T, kNormOne, 20, 128>(p, s);
  return norm_launch(rms_norm_long_kernel<T>, p.rows, 512, p, s);
}

template <typename T>
safe_status launch_rope(RopeParams& p, bool pairs, bool vec, cudaStream_t s) {
  constexpr int U = sizeof(T) == 2 ? 2 : 1;  // heads in flight for each lane
  if (vec) {
    // The ring for heads side by side in their rows and more tokens than its
    // CTAs take at once, from 4 KB a token in 16 bits: 51200 tokens of 24 + 24
    // heads of 96 take 152 us against 186 with plain loads, those of 8 + 2
    // heads of 128 (2.5 KB) 80 against 59. In fp32 lines are full either way:
    // 319 against 299 us.
    if constexpr (sizeof(T) == 2) {
      const size_t token = static_cast<size_t>(p.t[0].H + p.t[1].H) * p.d * sizeof(T);
      bool ring = token >= 4096 && token <= kRopeBulkMax;
      for (const RopeTensor& t : p.t) ring = ring && (t.H <= 1 || (t.xh == p.d && t.oh == p.d));
      const size_t smem = kRopeStages * ((token + 127) / 128 * 128) + p.r * sizeof(float2) + kRopeStages * sizeof(uint64_t);
      const size_t per_sm = 220 * 1024 / (smem + 1024) < 8 ? 220 * 1024 / (smem + 1024) : 8;
      const unsigned ctas = static_cast<unsigned>(per_sm * device_sms());
      if (ring && p.rows >= 2 * ctas) {
        constexpr int limit = kRopeStages * kRopeBulkMax + 1024 * sizeof(float2) + 256;
        if (!(pairs ? allow_smem<rope_bulk_kernel<T, true>>(limit) : allow_smem<rope_bulk_kernel<T, false>>(limit)))
          return SAFE_ERR_CUDA;
        if (pairs) rope_bulk_kernel<T, true><<<ctas, 128, smem, s>>>(p);
        else rope_bulk_kernel<T, false><<<ctas, 128, smem, s>>>(p);
        return launch_status();
      }
    }
    // few tokens: as few warps for each as take its heads in one batch (2458
    // tokens of 24 + 24 heads: 14.3 us against 18.4 with one warp); many: one
    const int per = p.r / 16, batch = U * (per < 32 ? 32 / per : 1), H = p.t[0].H + p.t[1].H;
    p.warps = H <= batch || p.rows > 32u * device_sms() ? 1 : H <= 2 * batch ? 2 : 4;
    const unsigned tokens = kRopeWarps / p.warps, grid = (p.rows + tokens - 1) / tokens;
    const size_t cs = static_cast<size_t>(tokens) * (p.r / 2) * sizeof(float2);
    if (pairs) rope_vec_kernel<T, true, U><<<grid, 32 * kRopeWarps, cs, s>>>(p);
    else rope_vec_kernel<T, false, U><<<grid, 32 * kRopeWarps, cs, s>>>(p);
    return launch_status();
  }
  const unsigned grid = (p.rows + kRopeWarps - 1) / kRopeWarps;
  const size_t smem = static_cast<size_t>(kRopeWarps) * (p.r / 2) * sizeof(float2);
  if (pairs) rope_kernel<T, true><<<grid, 32 * kRopeWarps, smem, s>>>(p);
  else rope_kernel<T, false><<<grid, 32 * kRopeWarps, smem, s>>>(p);
  return launch_status();
}

// Calls launch(first row, rows, positions) over slices of whole 128-row groups
// whose positions (a quarter of the rows times upr) stay below 2^31.
template <typename F>
safe_status mx_slices(int64_t rows, int upr, F launch) {
  const int64_t groups = (rows + 127) / 128, per = ((1ll << 31) - 256) / (32ll * upr);
  for (int64_t g = 0; g < groups; g += per) {
    const int64_t n = groups - g < per ? groups - g : per;
    launch(static_cast<int>(128 * g), static_cast<uint32_t>(n * 32 * upr));
    const safe_status st = launch_status();
    if (st != SAFE_OK) return st;
  }
  return SAFE_OK;
}

template <typename T>
safe_status launch_mx_quantize(MxQuantParams& p, int fmt, cudaStream_t s) {
  return mx_slices(p.rows, p.upr, [&](int row0, uint32_t threads) {
    p.row0 = row0;
    p.threads = threads;
    const unsigned blocks = (threads + 255) / 256;
    if (fmt == SAFE_MXFP8) mx_quantize_kernel<T, kMxFp8><<<blocks, 256, 0, s>>>(p);
    else if (fmt == SAFE_MXFP4) mx_quantize_kernel<T, kMxFp4><<<blocks, 256, 0, s>>>(p);
    else mx_quantize_kernel<T, kNvFp4><<<blocks, 256, 0, s>>>(p);
  });
}

template <typename T>
safe_status launch_mx_dequantize(MxDecodeParams& p, int fmt, cudaStream_t s) {
  return mx_slices(p.rows, p.upr, [&](int row0, uint32_t threads) {
    p.row0 = row0;
    p.threads = threads;
    const unsigned blocks = (threads + 255) / 256;
    if (fmt == SAFE_MXFP8) mx_dequantize_kernel<T, kMxFp8><<<blocks, 256, 0, s>>>(p);
    else if (fmt == SAFE_MXFP4) mx_dequantize_kernel<T, kMxFp4><<<blocks, 256, 0, s>>>(p);
    else mx_dequantize_kernel<T, kNvFp4><<<blocks, 256, 0, s>>>(p);
  });
}

// 2-D matrix [outer, inner] of bytes or 8-byte words (row pitch = inner); rows
// and columns past it read as zero.
bool encode_bytes_map(CUtensorMap* map, const void* base, bool words, uint64_t inner, uint64_t outer,
                      uint32_t box_inner, uint32_t box_outer) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * (words ? 8 : 1)};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t es[2] = {1, 1};
  return fn(map, words ? CU_TENSOR_MAP_DATA_TYPE_UINT64 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base),
            dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            words ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How many CTA pairs of a kernel can be resident at once on the current device.
template <auto kKernel>
int resident_pairs(int threads, int smem) {
  if (!allow_smem<kKernel>(smem)) return device_sms() / 2;
  static std::mutex mu;
  static int cached[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  const int sms = device_sms();
  std::lock_guard<std::mutex> lock(mu);
  int& n = cached[dev >= 0 && dev < 64 ? dev : 0];
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (sms / 2)));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    int c = 0;
    n = cudaOccupancyMaxActiveClusters(&c, kKernel, &cfg) == cudaSuccess && c > 0 ? c : sms / 2;
  }
  return n;
}

// How a microscaled layer's 256 x 256 tiles go over the resident CTA pairs: whole
// tiles in full waves, and those of the last, partial wave in pieces along
// d_in, as many as there are pairs for, whose fp32 sums a second kernel adds.
// The second launch costs what 12 stages do, the pieces' way through memory 28
// for 64 full pieces, so a split has to save more. Measured with / without
// (mxfp8, d_in 9216, d_out 2304): 2458 rows 49 / 57 us (90 tiles on 74 pairs, the
// last 16 in 4 pieces), 300 rows 25 / 33, 2 rows 16 / 29; where it would not
// pay, at an earlier step: 1000 rows (halves) 35 / 33, nvfp4 (half the stages) 2458 rows 35 / 34.
struct MxPlan {
  int pairs, n_tiles, rest, whole, split;
  int64_t units;
  size_t part_bytes;
};
MxPlan mx_linear_plan(int64_t M, int d_out, int row_bytes, int pairs, bool may_split) {
  MxPlan p{};
  p.pairs = pairs;
  p.n_tiles = (d_out + kMxTileN - 1) / kMxTileN;
  const int64_t tiles = (M + 255) / 256 * p.n_tiles;
  const int nk = (row_bytes + 127) / 128, rest = static_cast<int>(tiles % pairs);
  int split = rest > 0 ? pairs / rest : 1;
  if (split > nk / 4) split = nk / 4;  // pieces of four stages at least
  const int64_t row_tiles = (M + 255) / 256, rows = M / row_tiles;  // of a tile, on average
  const int64_t cost = 12 + 28 * rows * rest * split / (64 * 256);
  if (!may_split || split < 2 || nk - (nk + split - 1) / split <= cost || tiles > INT_MAX || rest * split > kMxPieces)
    split = 1;
  p.split = split;
  p.rest = split > 1 ? rest : 0;
  p.whole = static_cast<int>(tiles - p.rest);
  p.units = tiles - p.rest + static_cast<int64_t>(p.rest) * split;
  p.part_bytes = static_cast<size_t>(p.rest) * split * 256 * 256 * sizeof(float);
  return p;
}
int mx_linear_pairs(int fmt) {
  if (fmt == SAFE_MXFP8) return resident_pairs<mx_linear_pair_kernel<kMxFp8>>(kMxThreads, mx_linear_smem(kMxFp8));
  if (fmt == SAFE_MXFP4) return resident_pairs<mx_linear_pair_kernel<kMxFp4>>(kMxThreads, mx_linear_smem(kMxFp4));
  return resident_pairs<mx_linear_pair_kernel<kNvFp4>>(kMxThreads, mx_linear_smem(kNvFp4));
}

template <int kFmt>
safe_status launch_mx_linear(MxLinearParams& p, const void* X, const void* Xs, const void* W, const void* Ws, int d_in,
                             const MxPlan& plan, cudaStream_t s) {
  constexpr int smem = mx_linear_smem(kFmt), words = 64 * mx_stage_tiles(kFmt);
  const uint64_t ct = static_cast<uint64_t>(mx_tiles(d_in, kFmt)) * 64, rb = static_cast<uint64_t>(p.row_bytes);
  if (!encode_bytes_map(&p.x_map, X, false, rb, static_cast<uint64_t>(p.M), 128, 128) ||
      !encode_bytes_map(&p.w_map, W, false, rb, static_cast<uint64_t>(p.d_out), 128, 128) ||
      !encode_bytes_map(&p.xs_map, Xs, true, ct, static_cast<uint64_t>((p.M + 127LL) / 128), words, 1) ||
      !encode_bytes_map(&p.ws_map, Ws, true, ct, static_cast<uint64_t>((p.d_out + 127) / 128), words, 2))
    return SAFE_ERR_CUDA;
  if (!allow_smem<mx_linear_pair_kernel<kFmt>>(smem)) return SAFE_ERR_CUDA;
  const int pairs = p.units < plan.pairs ? p.units : plan.pairs;
  // both launches are programmatic dependents of what precedes them in the stream
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kMxThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, mx_linear_pair_kernel<kFmt>, p) != cudaSuccess) return SAFE_ERR_CUDA;
  if (plan.rest > 0) {
    const MxMergeParams m{p.part, p.bias, p.Y, p.alpha, p.M, p.d_out, p.act, p.n_tiles, p.whole, plan.split};
    cfg.gridDim = dim3(static_cast<unsigned>(32 * plan.rest));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, mx_linear_merge_kernel, m) != cudaSuccess) return SAFE_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace

extern "C" {

int safe_abi_version(void) { return kAbiVersion; }

const char* safe_status_string(int status) {
  switch (status) {
    case SAFE_OK: return "ok";
    case SAFE_ERR_INVALID_ARG: return "invalid argument";
    case SAFE_ERR_UNSUPPORTED: return "unsupported shape";
    case SAFE_ERR_CUDA: return "CUDA error";
    case SAFE_ERR_TIMEOUT: return "device wait timed out";
    case SAFE_ERR_DEVICE_CHECK: return "device-side input check failed";
    default: return "unknown status";
  }
}

safe_status safe_mask_classify(const void* mask, int dtype, const int64_t sizes[4], const int64_t strides[4],
                               int64_t* d_result, void* stream) {
  if (mask == nullptr || sizes == nullptr || strides == nullptr || d_result == nullptr) return SAFE_ERR_INVALID_ARG;
  if (dtype < SAFE_BOOL || dtype > SAFE_BF16) return SAFE_ERR_INVALID_ARG;
  for (int a = 0; a < 4; ++a)
    if (sizes[a] < 1 || strides[a] < 0) return SAFE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(d_result) & 7u) != 0) return SAFE_ERR_INVALID_ARG;
  const int esize = (dtype <= SAFE_U8) ? 1 : (dtype == SAFE_F32 ? 4 : 2);
  if ((reinterpret_cast<uintptr_t>(mask) % esize) != 0) return SAFE_ERR_INVALID_ARG;
  ClassifyParams p{};
  p.mask = static_cast<const uint8_t*>(mask);
  p.dtype = dtype;
  p.esize = esize;
  p.nb = strides[0] == 0 ? 1 : sizes[0];
  p.nh = strides[1] == 0 ? 1 : sizes[1];
  p.nq = strides[2] == 0 ? 1 : sizes[2];
  p.nk = strides[3] == 0 ? 1 : sizes[3];
  p.s0 = strides[0];
  p.s1 = strides[1];
  p.s2 = strides[2];
  p.s3 = strides[3];
  p.nfail = reinterpret_cast<unsigned long long*>(d_result + 1);
  p.first_fail = reinterpret_cast<unsigned long long*>(d_result + 2);
  cudaStream_t s = as_stream(stream);
  classify_init_kernel<<<1, 1, 0, s>>>(d_result);
  const int64_t rows = p.nb * p.nh * p.nq;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t want = (rows + 7) / 8;
  const int grid = static_cast<int>(want < static_cast<int64_t>(sms) * 16 ? want : static_cast<int64_t>(sms) * 16);
  classify_rows_kernel<<<grid, 256, 0, s>>>(p);
  classify_finalize_kernel<<<1, 1, 0, s>>>(d_result);
  return launch_status();
}

safe_status safe_mask_classify_sync(const void* mask, int dtype, const int64_t sizes[4], const int64_t strides[4],
                                    int64_t* d_result, int64_t* h_result, void* stream) {
  if (h_result == nullptr) return SAFE_ERR_INVALID_ARG;
  safe_status st = safe_mask_classify(mask, dtype, sizes, strides, d_result, stream);
  if (st != SAFE_OK) return st;
  cudaStream_t s = as_stream(stream);
  if (cudaMemcpyAsync(h_result, d_result, 3 * sizeof(int64_t), cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return SAFE_ERR_CUDA;
  return cudaStreamSynchronize(s) == cudaSuccess ? SAFE_OK : SAFE_ERR_CUDA;
}

size_t safe_attn_workspace_bytes(int B, int n_q, int N, int H, int d) {
  if (B < 1 || n_q < 1 || N < 1 || H < 1 || !supported_d(d)) return 0;
  return plan_flash(B, H, n_q, N, d, device_sms()).ws_bytes;
}

safe_status safe_attn_self(const void* Q, const void* K, const void* V, void* O, float* lse, int B, int N, int H,
                           int d, float scale, void* ws, size_t ws_bytes, void* stream) {
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return SAFE_ERR_INVALID_ARG;
  if (!sizes_ok(B, N, H) || !scale_ok(scale)) return SAFE_ERR_INVALID_ARG;
  if (!supported_d(d)) return SAFE_ERR_UNSUPPORTED;
  FlashParams p{};
  for (int c = 0; c < nchunks(d); ++c) {
    if (!encode_rows_map(&p.q_map[c], Q, B, N, H, d, c) || !encode_rows_map(&p.k_map[c], K, B, N, H, d, c) ||
        !encode_rows_map(&p.o_map[c], O, B, N, H, d, c))
      return SAFE_ERR_CUDA;
  }
  if (!encode_v_map(&p.v_map, V, B, N, H, d)) return SAFE_ERR_CUDA;
  p.S = nullptr;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.B = B;
  p.N = N;
  p.H = H;
  p.n_q = N;
  p.scale_log2 = scale * kLog2e;
  p.gather = 0;
  return dispatch_flash(d, p, ws, ws_bytes, as_stream(stream));
}

size_t safe_srsu_workspace_bytes(int B, int k, int N, int H, int d) {
  if (B < 1 || k < 1 || N < 1 || H < 1 || !supported_d(d)) return 0;
  return align256(safe_attn_workspace_bytes(B, k, N, H, d)) + static_cast<size_t>(B) * k * H * d * 2;
}

safe_status safe_srsu_attn(const void* Q, int q_compact, const int32_t* S, int k, const void* Kc, const void* Vc,
                           void* O_S, float* lse, int B, int N, int H, int d, float scale, void* ws, size_t ws_bytes,
                           void* stream) {
  if (!aligned16(Q) || !aligned16(Kc) || !aligned16(Vc) || !aligned16(O_S)) return SAFE_ERR_INVALID_ARG;
  if (!sizes_ok(B, N, H) || k < 1 || k > N || !scale_ok(scale)) return SAFE_ERR_INVALID_ARG;
  if (!q_compact && S == nullptr) return SAFE_ERR_INVALID_ARG;
  if (!supported_d(d)) return SAFE_ERR_UNSUPPORTED;
  if (!srsu_compact_q(Q, q_compact, S, k, B, N, H, d, ws, ws_bytes, as_stream(stream))) return SAFE_ERR_CUDA;
  FlashParams p{};
  if (!fill_srsu(p, Q, q_compact, S, k, Kc, Vc, O_S, lse, B, N, H, d, scale)) return SAFE_ERR_CUDA;
  return dispatch_flash(d, p, ws, ws_bytes, as_stream(stream));
}

safe_status safe_srsu_attn_assembled(const void* Q, int q_compact, const int32_t* S, int k, const void* Kcur,
                                     const void* Vcur, int cur_compact, const void* Kc, const void* Vc, void* O_S,
                                     float* lse, int B, int N, int H, int d, float scale, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (!aligned16(Q) || !aligned16(Kc) || !aligned16(Vc) || !aligned16(O_S) || !aligned16(Kcur) ||
      !aligned16(Vcur) || S == nullptr)
    return SAFE_ERR_INVALID_ARG;
  if (!sizes_ok(B, N, H) || k < 1 || k > N || !scale_ok(scale)) return SAFE_ERR_INVALID_ARG;
  if (!supported_d(d)) return SAFE_ERR_UNSUPPORTED;
  if (!srsu_compact_q(Q, q_compact, S, k, B, N, H, d, ws, ws_bytes, as_stream(stream))) return SAFE_ERR_CUDA;
  FlashParams p{};
  if (!fill_srsu(p, Q, q_compact, S, k, Kc, Vc, O_S, lse, B, N, H, d, scale)) return SAFE_ERR_CUDA;
  p.k_cur = static_cast<const __nv_bfloat16*>(Kcur);
  p.v_cur = static_cast<const __nv_bfloat16*>(Vcur);
  p.cur_compact = cur_compact ? 1 : 0;
  return dispatch_flash(d, p, ws, ws_bytes, as_stream(stream), true);
}

safe_status safe_attn_cross(const void* Q, const int32_t* q_idx, int nq, const void* Ky, const void* Vy,
                            const int32_t* valid_len, void* O, int B, int N, int M, int H, int d, float scale,
                            void* stream) {
  if (!aligned16(Q) || !aligned16(Ky) || !aligned16(Vy) || !aligned16(O) || valid_len == nullptr)
    return SAFE_ERR_INVALID_ARG;
  if (!sizes_ok(B, N, H) || M < 1 || !scale_ok(scale)) return SAFE_ERR_INVALID_ARG;
  if (q_idx == nullptr ? nq != N : (nq < 1 || nq > N)) return SAFE_ERR_INVALID_ARG;
  if (!supported_d(d) || M > 256) return SAFE_ERR_UNSUPPORTED;
  CrossParams p;
  safe_status st = fill_cross(p, Q, q_idx, nq, Ky, Vy, valid_len, nullptr, O, nullptr, B, N, M, H, d, scale);
  if (st != SAFE_OK) return st;
  return dispatch_cross(d, p, as_stream(stream));
}

size_t safe_pcsp_workspace_bytes(int B, int N, int H) {
  if (B < 1 || N < 1 || H < 1) return 0;
  return static_cast<size_t>(B) * H * N * sizeof(float);
}

safe_status safe_topk_partition(const float* scores, int B, int N, int k, int32_t* S, int32_t* C, void* stream) {
  if (scores == nullptr || S == nullptr || B < 1 || N < 1 || k < 1 || k > N) return SAFE_ERR_INVALID_ARG;
  if (N <= kTopkSmemKeys) {
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [] {
      attr_err = cudaFuncSetAttribute(topk_partition_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kTopkSmemKeys * static_cast<int>(sizeof(uint32_t)));
    });
    if (attr_err != cudaSuccess) return SAFE_ERR_CUDA;
    topk_partition_kernel<true><<<B, kTopkThreads, N * sizeof(uint32_t), as_stream(stream)>>>(scores, N, k, S, C);
  } else {
    topk_partition_kernel<false><<<B, kTopkThreads, 0, as_stream(stream)>>>(scores, N, k, S, C);
  }
  return launch_status();
}

safe_status safe_pcsp_topk(const void* Q, const void* Ky, const int32_t* valid_len, const float* w, int B, int N,
                           int M, int H, int d, float scale, float* scores, int accumulate, int k, int32_t* S,
                           int32_t* C, void* ws, size_t ws_bytes, void* stream) {
  if (scores == nullptr || !sizes_ok(B, N, H) || k < 0 || k > N) return SAFE_ERR_INVALID_ARG;
  if (k > 0 && S == nullptr) return SAFE_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  if (Q != nullptr) {
    if (!aligned16(Q) || !aligned16(Ky) || valid_len == nullptr || M < 1 || !scale_ok(scale))
      return SAFE_ERR_INVALID_ARG;
    if (!supported_d(d) || M > 256) return SAFE_ERR_UNSUPPORTED;
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 ||
        ws_bytes < safe_pcsp_workspace_bytes(B, N, H))
      return SAFE_ERR_INVALID_ARG;
    CrossParams p;
    // The value operand is not read when only scores are produced (O = null).
    safe_status st = fill_cross(p, Q, nullptr, N, Ky, Ky, valid_len, w, nullptr, static_cast<float*>(ws), B, N, M,
                                H, d, scale);
    if (st != SAFE_OK) return st;
    st = dispatch_cross(d, p, s);
    if (st != SAFE_OK) return st;
    dim3 grid((N + 255) / 256, B);
    pcsp_reduce_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(ws), scores, B, H, N, accumulate ? 1 : 0);
    st = launch_status();
    if (st != SAFE_OK) return st;
  }
  if (k > 0) return safe_topk_partition(scores, B, N, k, S, C, stream);
  return SAFE_OK;
}

safe_status safe_attn_cross_pcsp(const void* Q, const void* Ky, const void* Vy, const int32_t* valid_len,
                                 const float* w, void* O, int B, int N, int M, int H, int d, float scale,
                                 float* scores, int accumulate, int k, int32_t* S, int32_t* C, void* ws,
                                 size_t ws_bytes, void* stream) {
  if (!aligned16(Q) || !aligned16(Ky) || !aligned16(Vy) || !aligned16(O) || valid_len == nullptr || scores == nullptr)
    return SAFE_ERR_INVALID_ARG;
  if (!sizes_ok(B, N, H) || M < 1 || !scale_ok(scale) || k < 0 || k > N || (k > 0 && S == nullptr))
    return SAFE_ERR_INVALID_ARG;
  if (!supported_d(d) || M > 256) return SAFE_ERR_UNSUPPORTED;
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < safe_pcsp_workspace_bytes(B, N, H))
    return SAFE_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  CrossParams p;
  // one pass over the queries: the output rows and, from the same
  // probabilities, the per-head score partials
  safe_status st = fill_cross(p, Q, nullptr, N, Ky, Vy, valid_len, w, O, static_cast<float*>(ws), B, N, M, H, d,
                              scale);
  if (st != SAFE_OK) return st;
  st = dispatch_cross(d, p, s);
  if (st != SAFE_OK) return st;
  pcsp_reduce_kernel<<<dim3((N + 255) / 256, B), 256, 0, s>>>(static_cast<const float*>(ws), scores, B, H, N,
                                                              accumulate ? 1 : 0);
  st = launch_status();
  if (st != SAFE_OK) return st;
  if (k > 0) return safe_topk_partition(scores, B, N, k, S, C, stream);
  return SAFE_OK;
}

safe_status safe_pcsp_topk_noalloc(const void* Q, const void* Ky, const int32_t* valid_len, const float* w, int B,
                                   int N, int M, int H, int d, float scale, float* scores, int accumulate, int k,
                                   int32_t* S, int32_t* C, void* stream) {
  void* ws = nullptr;
  size_t ws_bytes = 0;
  if (Q != nullptr) {
    if (B < 1 || N < 1 || H < 1) return SAFE_ERR_INVALID_ARG;
    const size_t need = safe_pcsp_workspace_bytes(B, N, H);
    if (need > sizeof(g_pcsp_noalloc_scratch)) return SAFE_ERR_UNSUPPORTED;  // B*H*N above 2^21
    const safe_status st = noalloc_scratch(&ws);
    if (st != SAFE_OK) return st;
    ws_bytes = sizeof(g_pcsp_noalloc_scratch);
  }
  // Every element of the [B, H, N] partial block is written by the scoring
  // kernel before the head sum reads it, so nothing needs clearing.
  return safe_pcsp_topk(Q, Ky, valid_len, w, B, N, M, H, d, scale, scores, accumulate, k, S, C, ws, ws_bytes,
                        stream);
}

safe_status safe_ctx_cache_scatter(const void* Ksrc, const void* Vsrc, int src_compact, const int32_t* S, int k,
                                   void* Kc, void* Vc, int B, int N, int H, int d, void* stream) {
  if (!aligned16(Ksrc) || !aligned16(Vsrc) || !aligned16(Kc) || !aligned16(Vc)) return SAFE_ERR_INVALID_ARG;
  if (!sizes_ok(B, N, H) || d < 8 || (d % 8) != 0) return SAFE_ERR_INVALID_ARG;
  if (S != nullptr && (k < 1 || k > N)) return SAFE_ERR_INVALID_ARG;
  if (S == nullptr && src_compact) return SAFE_ERR_INVALID_ARG;
  const int row_units = H * d * 2 / 16;
  const int64_t rows = S != nullptr ? static_cast<int64_t>(B) * k : static_cast<int64_t>(B) * N;
  const int64_t blocks = (rows * 32 + 255) / 256;
  if (blocks > INT_MAX) return SAFE_ERR_UNSUPPORTED;
  cache_scatter_kernel<<<static_cast<unsigned>(blocks), 256, 0, as_stream(stream)>>>(
      static_cast<const uint4*>(Ksrc), static_cast<const uint4*>(Vsrc), src_compact, S, k, static_cast<uint4*>(Kc),
      static_cast<uint4*>(Vc), B, N, row_units);
  return launch_status();
}

// ---------------------------------------------------------------- sensitivity field and SW-CFG
size_t safe_sensitivity_workspace_bytes(int B, int N) {
  if (B < 1 || N < 1) return 0;
  return align256(static_cast<size_t>(B) * N * sizeof(float)) + align256(static_cast<size_t>(B) * 2 * sizeof(uint32_t));
}

safe_status safe_sensitivity_field(const float* scores, float* s, int B, int grid_h, int grid_w, float sigma,
                                   float truncate, void* ws, size_t ws_bytes, void* stream) {
  if (scores == nullptr || s == nullptr || scores == s || B < 1 || B > 65535 || grid_h < 1 || grid_w < 1)
    return SAFE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(grid_h) * grid_w > INT_MAX / 2) return SAFE_ERR_INVALID_ARG;
  if (!std::isfinite(sigma) || sigma < 0.f || !std::isfinite(truncate) || truncate <= 0.f) return SAFE_ERR_INVALID_ARG;
  const int N = grid_h * grid_w;
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < safe_sensitivity_workspace_bytes(B, N))
    return SAFE_ERR_INVALID_ARG;
  SmoothParams p{};
  // the taps of G_sigma, in double, then rounded to fp32
  const double r_real = sigma > 0.f ? std::floor(static_cast<double>(truncate) * sigma + 0.5) : 0.0;
  if (r_real > kMaxSmoothRadius) return SAFE_ERR_UNSUPPORTED;
  p.r = static_cast<int>(r_real);
  if (p.r == 0) {
    p.taps[0] = 1.f;
  } else {
    double g[kMaxTaps], sum = 0.0;
    for (int t = -p.r; t <= p.r; ++t) {
      g[t + p.r] = std::exp(-(static_cast<double>(t) * t) / (2.0 * sigma * sigma));
      sum += g[t + p.r];
    }
    for (int t = 0; t <= 2 * p.r; ++t) p.taps[t] = static_cast<float>(g[t] / sum);
  }
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.in = scores;
  p.rows = reinterpret_cast<float*>(w);
  p.out = s;
  p.minmax = reinterpret_cast<uint32_t*>(w + align256(static_cast<size_t>(B) * N * sizeof(float)));
  p.B = B;
  p.gh = grid_h;
  p.gw = grid_w;
  cudaStream_t st = as_stream(stream);
  const dim3 grid((N + 255) / 256, B);
  smooth_rows_kernel<<<grid, 256, 0, st>>>(p);
  smooth_cols_kernel<<<grid, 256, 0, st>>>(p);
  norm01_kernel<<<grid, 256, 0, st>>>(s, p.minmax, N);
  return launch_status();
}

// ---------------------------------------------------------------- row-wise layers of the block
size_t safe_gather_linear_workspace_bytes(int B, int k, int d_in) {
  if (B < 1 || k < 1 || d_in < 1) return 0;
  return static_cast<size_t>(B) * k * d_in * 2;
}

safe_status safe_gather_linear(const void* X, const int32_t* S, int k, const void* Wt, const float* bias, int act,
                               void* Y, int B, int N, int d_in, int d_out, void* ws, size_t ws_bytes, void* stream) {
  if (!aligned16(X) || !aligned16(Wt) || !aligned16(Y)) return SAFE_ERR_INVALID_ARG;
  if (bias != nullptr && (reinterpret_cast<uintptr_t>(bias) & 3u) != 0) return SAFE_ERR_INVALID_ARG;
  if (!sizes_ok(B, N, 1) || (S != nullptr && (k < 1 || k > N))) return SAFE_ERR_INVALID_ARG;
  if (d_in < 64 || d_in % 8 != 0 || d_out < 8 || d_out % 8 != 0 || (act != 0 && act != 1)) return SAFE_ERR_INVALID_ARG;
  if (S != nullptr && aligned16(ws) && ws_bytes >= safe_gather_linear_workspace_bytes(B, k, d_in)) {
    // the rows of S as a compact [B, k, d_in] matrix, then the GEMM over
    // every row of it (tiled operand copies instead of per-row gathers)
    const long long rows = static_cast<long long>(B) * k;
    if ((rows + 7) / 8 > INT_MAX) return SAFE_ERR_UNSUPPORTED;
    gather_rows_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, as_stream(stream)>>>(
        static_cast<const uint4*>(X), S, static_cast<uint4*>(ws), B, N, k, d_in / 8);
    if (cudaGetLastError() != cudaSuccess) return SAFE_ERR_CUDA;
    X = ws;
    N = k;
    S = nullptr;
  }
  const int R = S != nullptr ? k : N;
  // plain rows: CTA pairs on 256 x 256 tiles; rows of S gathered in the
  // kernel (no workspace): one CTA per 128 x 256 tile
  const bool pairs = S == nullptr;
  const int64_t m_tiles = (R + (pairs ? 255 : 127)) / (pairs ? 256 : 128), n_tiles = (d_out + 255) / 256;
  const int64_t tiles = static_cast<int64_t>(B) * m_tiles * n_tiles;
  if (tiles > INT_MAX) return SAFE_ERR_UNSUPPORTED;
  LinearParams p{};
  if (!encode_matrix_map(&p.x_map, X, static_cast<uint64_t>(d_in), static_cast<uint64_t>(B) * N, 64, 1) ||
      !encode_matrix_map(&p.xt_map, X, static_cast<uint64_t>(d_in), static_cast<uint64_t>(B) * N, 64, 128) ||
      !encode_matrix_map(&p.w_map, Wt, static_cast<uint64_t>(d_in), static_cast<uint64_t>(d_out), 64, 256) ||
      !encode_matrix_map(&p.w2_map, Wt, static_cast<uint64_t>(d_in), static_cast<uint64_t>(d_out), 64, 128))
    return SAFE_ERR_CUDA;
  p.S = S;
  p.bias = bias;
  p.Y = static_cast<__nv_bfloat16*>(Y);
  p.B = B;
  p.N = N;
  p.R = R;
  p.d_in = d_in;
  p.d_out = d_out;
  p.act = act;
  p.m_tiles = static_cast<int>(m_tiles);
  p.n_tiles = static_cast<int>(n_tiles);
  p.tiles = static_cast<int>(tiles);
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(linear_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinSmem);
    if (attr_err == cudaSuccess)
      attr_err = cudaFuncSetAttribute(linear_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLin2Smem);
  });
  if (attr_err != cudaSuccess) return SAFE_ERR_CUDA;
  const int sms = device_sms();
  if (pairs) {
    // as many pairs as can be resident at once (a GPC with an odd number of
    // free SMs leaves one of them out), so that every pair starts at once
    static int max_pairs[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    int& mp = max_pairs[dev >= 0 && dev < 64 ? dev : 0];
    if (mp == 0) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(2 * (sms / 2)));
      cfg.blockDim = dim3(kLinThreads);
      cfg.dynamicSmemBytes = kLin2Smem;
      int n = 0;
      mp = cudaOccupancyMaxActiveClusters(&n, linear_pair_kernel, &cfg) == cudaSuccess && n > 0 ? n : sms / 2;
    }
    const int n_pairs = static_cast<int>(tiles < mp ? tiles : mp);
    linear_pair_kernel<<<2 * (n_pairs > 0 ? n_pairs : 1), kLinThreads, kLin2Smem, as_stream(stream)>>>(p);
  } else {
    const int grid = static_cast<int>(tiles < sms ? tiles : sms);
    linear_kernel<<<grid, kLinThreads, kLinSmem, as_stream(stream)>>>(p);
  }
  return launch_status();
}

// ---------------------------------------------------------------- norm, positions, microscaled layers
size_t safe_mx_scale_bytes(int64_t rows, int D, int fmt) {
  if (rows < 1 || D < 1 || D % 32 != 0 || fmt < SAFE_MXFP8 || fmt > SAFE_NVFP4) return 0;
  return static_cast<size_t>((rows + 127) / 128) * mx_tiles(D, fmt) * 512;
}

safe_status safe_rms_norm(const void* x, int x_full, const void* res, const int32_t* S, int k, const float* w,
                          float eps, void* h, int h_full, void* y, void* q, void* q_scales, int dtype, int B, int N,
                          int D, void* stream) {
  const size_t e = float_size(dtype);
  if (e == 0) return SAFE_ERR_UNSUPPORTED;
  if (!sizes_ok(B, N, 1) || D < 1 || (S != nullptr && (k < 1 || k > N))) return SAFE_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return SAFE_ERR_INVALID_ARG;
  if (x == nullptr || (y == nullptr && q == nullptr) || (q == nullptr) != (q_scales == nullptr)) return SAFE_ERR_INVALID_ARG;
  if (S == nullptr && (x_full || h_full)) return SAFE_ERR_INVALID_ARG;
  if (h_full && (res == nullptr || h != res)) return SAFE_ERR_INVALID_ARG;  // the rows S of the stream, in place
  if (!aligned_to(x, e) || !aligned_to(res, e) || !aligned_to(S, 4) || !aligned_to(w, 4) || !aligned_to(h, e) ||
      !aligned_to(y, e))
    return SAFE_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(q_scales, 16)) return SAFE_ERR_INVALID_ARG;
  const int R = S != nullptr ? k : N;
  NormParams p{};
  p.rows = B * R;  // <= B N <= INT_MAX
  // room for the counters past the last row and element
  if (p.rows > INT_MAX - 511 || D > INT_MAX - 511) return SAFE_ERR_UNSUPPORTED;
  const size_t n_full = static_cast<size_t>(B) * N * D, n_rows = static_cast<size_t>(p.rows) * D;
  // outputs apart from each other and from the inputs; without S, h and y may
  // take the place of x or res (each row is read before it is written)
  const size_t xb = (x_full ? n_full : n_rows) * e, rb = n_full * e, ob = n_rows * e;
  const size_t sb = q != nullptr ? safe_mx_scale_bytes(p.rows, D, SAFE_MXFP8) : 0;
  auto clash = [&](const void* o, size_t obytes, const void* in, size_t ibytes) {
    return overlap(o, obytes, in, ibytes) && !(S == nullptr && o == in);
  };
  if (clash(y, ob, x, xb) || clash(y, ob, res, rb) || clash(h, h_full ? 0 : ob, x, xb) ||
      clash(h, h_full ? 0 : ob, res, rb) || overlap(h, h_full ? rb : ob, y, ob) || (h_full && overlap(h, rb, x, xb)))
    return SAFE_ERR_INVALID_ARG;
  const size_t hb = h_full ? rb : ob, wb = static_cast<size_t>(D) * 4, Sb = static_cast<size_t>(p.rows) * 4;
  if (overlap(y, ob, w, wb) || overlap(h, hb, w, wb) || overlap(y, ob, S, Sb) || overlap(h, hb, S, Sb))
    return SAFE_ERR_INVALID_ARG;
  if (q != nullptr) {
    const void* in[] = {x, res, S, w, h, y};
    const size_t len[] = {xb, rb, Sb, wb, hb, ob};
    for (int i = 0; i < 6; ++i)
      if (overlap(q, n_rows, in[i], len[i]) || overlap(q_scales, sb, in[i], len[i])) return SAFE_ERR_INVALID_ARG;
    if (overlap(q, n_rows, q_scales, sb)) return SAFE_ERR_INVALID_ARG;
  }
  const bool aligned = aligned_to(x, 16) && aligned_to(res, 16) && aligned_to(h, 16) && aligned_to(y, 16);
  const bool vec = aligned && D % 8 == 0 && aligned_to(w, 16);
  const int mode = vec ? kNormVec : aligned && S == nullptr ? kNormShift : kNormOne;
  if (q != nullptr && (D % 32 != 0 || !vec)) return SAFE_ERR_INVALID_ARG;
  if (q != nullptr && D > kNormMaxVec) return SAFE_ERR_UNSUPPORTED;
  p.x = x;
  p.res = res;
  p.S = S;
  p.w = w;
  p.h = h;
  p.y = y;
  p.q = static_cast<uint8_t*>(q);
  p.q_scales = static_cast<uint8_t*>(q_scales);
  p.eps = eps;
  p.N = N;
  p.R = R;
  p.D = D;
  p.x_full = x_full ? 1 : 0;
  p.h_full = h_full ? 1 : 0;
  p.ct = q != nullptr ? mx_tiles(D, SAFE_MXFP8) : 0;
  p.rows_pad = q != nullptr ? (p.rows + 127) / 128 * 128 : p.rows;
  p.inv_D = 1.f / static_cast<float>(D);
  p.by_R = fast_div(static_cast<uint32_t>(R > 1 ? R : 2));
  if (h_full && R > 1) {
    uint8_t* mark = static_cast<uint8_t*>(y != nullptr ? y : q);
    p.mark = mark;
    p.mark_pitch = static_cast<size_t>(D) * (y != nullptr ? e : 1);
    const unsigned tiles = (static_cast<unsigned>(R) + 1023u) / 1024u;
    const unsigned per = (tiles + kNormOrderCtas - 1) / kNormOrderCtas, ctas = (tiles + per - 1) / per;
    norm_order_kernel<<<dim3(ctas, static_cast<unsigned>(B)), 1024, 0, as_stream(stream)>>>(
        S, static_cast<uint32_t>(R), 1024 * per, mark, p.mark_pitch);
    const safe_status st = launch_status();
    if (st != SAFE_OK) return st;
  }
  switch (dtype) {
    case SAFE_F32: return launch_norm<float>(p, mode, as_stream(stream));
    case SAFE_F16: return launch_norm<__half>(p, mode, as_stream(stream));
    default: return launch_norm<__nv_bfloat16>(p, mode, as_stream(stream));
  }
}

safe_status safe_rope(const void* q, const int64_t q_strides[3], void* oq, const int64_t oq_strides[3], int Hq,
                      const void* k, const int64_t k_strides[3], void* ok, const int64_t ok_strides[3], int Hk,
                      int dtype, const int64_t* freq, const int32_t* sections, int axes, const int32_t* pos,
                      int pos_batched, const int32_t* S, int B, int N, int R, int d, int r, int interleaved, float m,
                      void* stream) {
  const size_t e = float_size(dtype);
  if (e == 0) return SAFE_ERR_UNSUPPORTED;
  if (q == nullptr || oq == nullptr || Hq < 1) return SAFE_ERR_INVALID_ARG;
  if (k == nullptr ? (ok != nullptr || Hk != 0) : (ok == nullptr || Hk < 1)) return SAFE_ERR_INVALID_ARG;
  if (!sizes_ok(B, N, Hq) || Hk > 65535 || R < 1 || R > N || (S == nullptr && R != N)) return SAFE_ERR_INVALID_ARG;
  if (d < 2 || r < 2 || r > d || r % 2 != 0 || freq == nullptr || sections == nullptr || !std::isfinite(m))
    return SAFE_ERR_INVALID_ARG;
  if (axes < 1 || axes > 3 || (pos == nullptr && axes != 1)) return SAFE_ERR_INVALID_ARG;
  if (d > 1024) return SAFE_ERR_UNSUPPORTED;
  int sum = 0;
  for (int a = 0; a < axes; ++a) {
    if (sections[a] < 0 || sections[a] > r / 2) return SAFE_ERR_INVALID_ARG;
    sum += sections[a];
  }
  if (sum != r / 2) return SAFE_ERR_INVALID_ARG;
  if (!aligned_to(freq, 8) || !aligned_to(pos, 4) || !aligned_to(S, 4)) return SAFE_ERR_INVALID_ARG;
  RopeParams p{};
  bool vec = d % 8 == 0 && r % 16 == 0;
  const void* xs[2] = {q, k};
  void* os[2] = {oq, ok};
  const int64_t q_own[3] = {static_cast<int64_t>(R) * Hq * d, static_cast<int64_t>(Hq) * d, d};
  const int64_t k_own[3] = {static_cast<int64_t>(R) * Hk * d, static_cast<int64_t>(Hk) * d, d};
  const int64_t* st[4] = {q_strides ? q_strides : q_own, oq_strides ? oq_strides : q_own, k_strides ? k_strides : k_own,
                          ok_strides ? ok_strides : k_own};
  const int heads[2] = {Hq, Hk}, n = k != nullptr ? 2 : 1;
  View4 in[2], out[2];
  bool in_place[2] = {};
  for (int i = 0; i < n; ++i) {
    RopeTensor& t = p.t[i];
    if (!aligned_to(xs[i], e) || !aligned_to(os[i], e)) return SAFE_ERR_INVALID_ARG;
    for (int a = 0; a < 3; ++a) {
      if (st[2 * i][a] < 0 || st[2 * i + 1][a] < 0) return SAFE_ERR_INVALID_ARG;
      vec = vec && st[2 * i][a] % 8 == 0 && st[2 * i + 1][a] % 8 == 0;
    }
    const int64_t* o = st[2 * i + 1];
    vec = vec && aligned_to(xs[i], 16) && aligned_to(os[i], 16);
    t = RopeTensor{xs[i], os[i], st[2 * i][0], st[2 * i][1], st[2 * i][2], o[0], o[1], o[2], heads[i]};
    in[i] = View4{reinterpret_cast<uintptr_t>(xs[i]), {B, R, heads[i]}, {t.xb, t.xn, t.xh}, d};
    out[i] = View4{reinterpret_cast<uintptr_t>(os[i]), {B, R, heads[i]}, {t.ob, t.on, t.oh}, d};
    if (!nested(d, out[i].size, out[i].stride, 3)) return SAFE_ERR_INVALID_ARG;
    in_place[i] = xs[i] == os[i] && t.xb == t.ob && t.xn == t.on && t.xh == t.oh;
    if (!in_place[i]) p.copy_tail = r < d;
  }
  // an output shares no element with the other one, nor with an input that is not its own in place
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      if ((i != j || !in_place[i]) && !apart(out[i], in[j], e)) return SAFE_ERR_INVALID_ARG;
  if (n == 2 && !apart(out[0], out[1], e)) return SAFE_ERR_INVALID_ARG;
  // nor with freq, pos or S
  for (int i = 0; i < n; ++i) {
    const size_t ob = static_cast<size_t>(extent(out[i], true, true)) * e;
    if (overlap(os[i], ob, freq, static_cast<size_t>(r / 2) * 8) ||
        overlap(os[i], ob, pos, static_cast<size_t>(pos_batched ? B : 1) * N * axes * 4) ||
        overlap(os[i], ob, S, static_cast<size_t>(B) * R * 4))
      return SAFE_ERR_INVALID_ARG;
  }
  p.freq = reinterpret_cast<const long long*>(freq);
  p.pos = pos;
  p.pos_b = pos_batched ? static_cast<long long>(N) * axes : 0;
  p.S = S;
  p.axes = axes;
  p.sec0 = sections[0];
  p.sec1 = axes > 1 ? sections[1] : 0;
  p.N = N;
  p.R = R;
  p.d = d;
  p.r = r;
  p.m = m;
  p.rows = static_cast<uint32_t>(B) * R;  // <= B N <= INT_MAX
  cudaStream_t s = as_stream(stream);
  switch (dtype) {
    case SAFE_F32: return launch_rope<float>(p, interleaved != 0, vec, s);
    case SAFE_F16: return launch_rope<__half>(p, interleaved != 0, vec, s);
    default: return launch_rope<__nv_bfloat16>(p, interleaved != 0, vec, s);
  }
}

safe_status safe_mx_quantize(const void* X, int dtype, const int32_t* S, int k, int fmt, float g, void* data,
                             void* scales, int B, int N, int D, void* stream) {
  if (float_size(dtype) == 0) return SAFE_ERR_UNSUPPORTED;
  if (!aligned16(X) || !aligned16(data) || !aligned16(scales) || !aligned_to(S, 4)) return SAFE_ERR_INVALID_ARG;
  if (!sizes_ok(B, N, 1) || (S != nullptr && (k < 1 || k > N)) || D < 32 || D % 32 != 0) return SAFE_ERR_INVALID_ARG;
  if (!mx_factor_ok(fmt, g)) return SAFE_ERR_INVALID_ARG;
  if (D > kMxMaxD || static_cast<int64_t>(B) * (S != nullptr ? k : N) > kMxMaxRows) return SAFE_ERR_UNSUPPORTED;
  MxQuantParams p{};
  p.X = X;
  p.S = S;
  p.data = static_cast<uint8_t*>(data);
  p.scales = static_cast<uint8_t*>(scales);
  p.g = g;
  p.inv6g = 1.f / (6.f * g);
  p.N = N;
  p.R = S != nullptr ? k : N;
  p.D = D;
  p.ct = mx_tiles(D, fmt);
  p.upr = p.ct * 4 * (fmt == SAFE_NVFP4 ? 1 : 2);
  p.rows = B * p.R;  // <= B N <= INT_MAX
  p.wide = aligned_to(X, 32);
  p.by_upr = fast_div(static_cast<uint32_t>(p.upr));
  p.by_R = fast_div(static_cast<uint32_t>(p.R > 1 ? p.R : 2));
  const size_t db = static_cast<size_t>(p.rows) * (fmt == SAFE_MXFP8 ? D : D / 2);
  const size_t sb = safe_mx_scale_bytes(p.rows, D, fmt), xb = static_cast<size_t>(B) * N * D * float_size(dtype);
  if (overlap(data, db, X, xb) || overlap(scales, sb, X, xb) || overlap(data, db, scales, sb)) return SAFE_ERR_INVALID_ARG;
  const size_t Sb = static_cast<size_t>(p.rows) * 4;
  if (overlap(data, db, S, Sb) || overlap(scales, sb, S, Sb)) return SAFE_ERR_INVALID_ARG;
  switch (dtype) {
    case SAFE_F32: return launch_mx_quantize<float>(p, fmt, as_stream(stream));
    case SAFE_F16: return launch_mx_quantize<__half>(p, fmt, as_stream(stream));
    default: return launch_mx_quantize<__nv_bfloat16>(p, fmt, as_stream(stream));
  }
}

safe_status safe_mx_dequantize(const void* data, const void* scales, int fmt, float g, void* Y, int dtype,
                               int64_t rows, int D, void* stream) {
  if (float_size(dtype) == 0) return SAFE_ERR_UNSUPPORTED;
  if (!aligned16(data) || !aligned16(scales) || !aligned16(Y)) return SAFE_ERR_INVALID_ARG;
  if (rows < 1 || rows > INT_MAX || D < 32 || D % 32 != 0 || !mx_factor_ok(fmt, g)) return SAFE_ERR_INVALID_ARG;
  if (D > kMxMaxD || rows > kMxMaxRows) return SAFE_ERR_UNSUPPORTED;
  const size_t db = static_cast<size_t>(rows) * (fmt == SAFE_MXFP8 ? D : D / 2);
  const size_t yb = static_cast<size_t>(rows) * D * float_size(dtype);
  if (overlap(Y, yb, data, db) || overlap(Y, yb, scales, safe_mx_scale_bytes(rows, D, fmt))) return SAFE_ERR_INVALID_ARG;
  MxDecodeParams p{};
  p.data = static_cast<const uint8_t*>(data);
  p.scales = static_cast<const uint8_t*>(scales);
  p.Y = Y;
  p.g = g;
  p.D = D;
  p.ct = mx_tiles(D, fmt);
  p.upr = D / 16;
  p.rows = static_cast<int>(rows);
  p.wide = aligned_to(Y, 32);
  p.by_upr = fast_div(static_cast<uint32_t>(p.upr));
  switch (dtype) {
    case SAFE_F32: return launch_mx_dequantize<float>(p, fmt, as_stream(stream));
    case SAFE_F16: return launch_mx_dequantize<__half>(p, fmt, as_stream(stream));
    default: return launch_mx_dequantize<__nv_bfloat16>(p, fmt, as_stream(stream));
  }
}

size_t safe_mx_linear_workspace_bytes(int64_t rows, int d_in, int d_out, int fmt) {
  if (fmt < SAFE_MXFP8 || fmt > SAFE_NVFP4 || rows < 1 || rows > kMxMaxRows || d_in < 64 || d_in > kMxMaxD ||
      d_in % 32 != 0 || d_out < 8 || d_out > kMxMaxRows || d_out % 8 != 0)
    return 0;
  return mx_linear_plan(rows, d_out, fmt == SAFE_MXFP8 ? d_in : d_in / 2, mx_linear_pairs(fmt), true).part_bytes;
}

safe_status safe_mx_linear(const void* X, const void* X_scales, const void* Wt, const void* Wt_scales, int fmt,
                           float alpha, const float* bias, int act, void* Y, int64_t rows, int d_in, int d_out,
                           void* ws, size_t ws_bytes, void* stream) {
  if (!aligned16(X) || !aligned16(X_scales) || !aligned16(Wt) || !aligned16(Wt_scales) || !aligned16(Y) ||
      !aligned_to(bias, 4))
    return SAFE_ERR_INVALID_ARG;
  if (fmt < SAFE_MXFP8 || fmt > SAFE_NVFP4 || !std::isnormal(alpha) || (act != 0 && act != 1)) return SAFE_ERR_INVALID_ARG;
  if (rows < 1 || rows > INT_MAX || d_in < 64 || d_in % 32 != 0 || d_out < 8 || d_out % 8 != 0) return SAFE_ERR_INVALID_ARG;
  // a tile's stages, which the epilogue waits for at once, take 3 ms at the largest d_in
  if (rows > kMxMaxRows || d_out > kMxMaxRows || d_in > kMxMaxD) return SAFE_ERR_UNSUPPORTED;
  const int row_bytes = fmt == SAFE_MXFP8 ? d_in : d_in / 2;
  const size_t yb = static_cast<size_t>(rows) * d_out * 2;
  if (overlap(Y, yb, X, static_cast<size_t>(rows) * row_bytes) ||
      overlap(Y, yb, X_scales, safe_mx_scale_bytes(rows, d_in, fmt)) ||
      overlap(Y, yb, Wt, static_cast<size_t>(d_out) * row_bytes) ||
      overlap(Y, yb, Wt_scales, safe_mx_scale_bytes(d_out, d_in, fmt)) ||
      overlap(Y, yb, bias, static_cast<size_t>(d_out) * 4))
    return SAFE_ERR_INVALID_ARG;
  const int pairs = mx_linear_pairs(fmt);
  MxPlan plan = mx_linear_plan(rows, d_out, row_bytes, pairs, ws != nullptr);
  if (plan.part_bytes > 0) {
    if (ws_bytes < plan.part_bytes) {
      plan = mx_linear_plan(rows, d_out, row_bytes, pairs, false);
    } else if (!aligned_to(ws, 32) || overlap(ws, plan.part_bytes, Y, yb) ||
               overlap(ws, plan.part_bytes, X, static_cast<size_t>(rows) * row_bytes) ||
               overlap(ws, plan.part_bytes, X_scales, safe_mx_scale_bytes(rows, d_in, fmt)) ||
               overlap(ws, plan.part_bytes, Wt, static_cast<size_t>(d_out) * row_bytes) ||
               overlap(ws, plan.part_bytes, Wt_scales, safe_mx_scale_bytes(d_out, d_in, fmt)) ||
               overlap(ws, plan.part_bytes, bias, static_cast<size_t>(d_out) * 4)) {
      return SAFE_ERR_INVALID_ARG;
    }
  }
  if (plan.units > INT_MAX) return SAFE_ERR_UNSUPPORTED;
  MxLinearParams p{};
  p.n_tiles = plan.n_tiles;
  p.whole = plan.whole;
  for (int t = 0; t < plan.rest; ++t)
    for (int k = 0, nk = (row_bytes + 127) / 128; k < plan.split; ++k) {
      const int i = t * plan.split + k, k0 = nk * k / plan.split;
      p.piece_tile[i] = static_cast<uint16_t>(t);
      p.piece_k0[i] = static_cast<uint16_t>(k0);
      p.piece_n[i] = static_cast<uint16_t>(nk * (k + 1) / plan.split - k0);
    }
  p.units = static_cast<int>(plan.units);
  p.part = static_cast<float*>(ws);
  p.bias = bias;
  p.Y = static_cast<__nv_bfloat16*>(Y);
  p.wide = d_out % 16 == 0 && aligned_to(Y, 32);
  p.alpha = alpha;
  p.M = static_cast<int>(rows);
  p.row_bytes = row_bytes;
  p.d_out = d_out;
  p.act = act;
  switch (fmt) {
    case SAFE_MXFP8: return launch_mx_linear<kMxFp8>(p, X, X_scales, Wt, Wt_scales, d_in, plan, as_stream(stream));
    case SAFE_MXFP4: return launch_mx_linear<kMxFp4>(p, X, X_scales, Wt, Wt_scales, d_in, plan, as_stream(stream));
    default: return launch_mx_linear<kNvFp4>(p, X, X_scales, Wt, Wt_scales, d_in, plan, as_stream(stream));
  }
}

safe_status safe_partition_indicator(const int32_t* S, int k, float* s, int B, int N, void* stream) {
  if (S == nullptr || s == nullptr || B < 1 || B > 65535 || N < 1 || k < 1 || k > N) return SAFE_ERR_INVALID_ARG;
  partition_indicator_kernel<<<dim3((N + 255) / 256, B), 256, 0, as_stream(stream)>>>(S, k, s, N);
  return launch_status();
}

safe_status safe_sw_cfg(const void* f_c, const void* f_u, const float* s, void* out, int dtype, int B, int N, int C,
                        float gamma_ctx, float gamma_sens, void* stream) {
  if (f_c == nullptr || f_u == nullptr || s == nullptr || out == nullptr || B < 1 || N < 1 || C < 1)
    return SAFE_ERR_INVALID_ARG;
  if (dtype != SAFE_F32 && dtype != SAFE_BF16) return SAFE_ERR_UNSUPPORTED;
  if (!std::isfinite(gamma_ctx) || !std::isfinite(gamma_sens)) return SAFE_ERR_INVALID_ARG;
  const size_t esize = dtype == SAFE_F32 ? 4 : 2;
  auto aligned = [](const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; };
  if (!aligned(f_c, esize) || !aligned(f_u, esize) || !aligned(out, esize) || !aligned(s, 4))
    return SAFE_ERR_INVALID_ARG;
  const size_t total = static_cast<size_t>(B) * N * C;
  const int vec = static_cast<int>(16 / esize);
  const bool vec_ok = (C % vec) == 0 && aligned(f_c, 16) && aligned(f_u, 16) && aligned(out, 16);
  const size_t n_vec = vec_ok ? total / vec : total;
  const size_t want = (n_vec + 255) / 256;
  const unsigned blocks = static_cast<unsigned>(want < static_cast<size_t>(device_sms()) * 16 ? (want ? want : 1)
                                                                                          : static_cast<size_t>(device_sms()) * 16);
  const float diff = gamma_sens - gamma_ctx;
  cudaStream_t st = as_stream(stream);
  if (dtype == SAFE_F32) {
    auto fc = static_cast<const float*>(f_c);
    auto fu = static_cast<const float*>(f_u);
    auto o = static_cast<float*>(out);
    if (vec_ok) sw_cfg_kernel<float, 4><<<blocks, 256, 0, st>>>(fc, fu, s, o, n_vec, C, gamma_ctx, diff);
    else sw_cfg_kernel<float, 1><<<blocks, 256, 0, st>>>(fc, fu, s, o, n_vec, C, gamma_ctx, diff);
  } else {
    auto fc = static_cast<const __nv_bfloat16*>(f_c);
    auto fu = static_cast<const __nv_bfloat16*>(f_u);
    auto o = static_cast<__nv_bfloat16*>(out);
    if (vec_ok) sw_cfg_kernel<__nv_bfloat16, 8><<<blocks, 256, 0, st>>>(fc, fu, s, o, n_vec, C, gamma_ctx, diff);
    else sw_cfg_kernel<__nv_bfloat16, 1><<<blocks, 256, 0, st>>>(fc, fu, s, o, n_vec, C, gamma_ctx, diff);
  }
  return launch_status();
}

safe_status safe_get_device_status(int* h_status, void* stream) {
  if (h_status == nullptr) return SAFE_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return SAFE_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int)) != cudaSuccess) return SAFE_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) != cudaSuccess) return SAFE_ERR_CUDA;
  *h_status = v;
  return SAFE_OK;
}

safe_status safe_selftest_wait_timeout(uint64_t limit_ns, void* stream) {
  if (limit_ns == 0 || limit_ns > 1000000000ull) return SAFE_ERR_INVALID_ARG;
  selftest_wait_kernel<<<1, 32, 0, as_stream(stream)>>>(limit_ns);
  return launch_status();
}

}  // extern "C"
